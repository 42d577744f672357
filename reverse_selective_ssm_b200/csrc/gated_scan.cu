// Entry points of the gated linear recurrence: r2l_gated_scan and its training
// forward.
#include <type_traits>

#include "gated_host.cuh"

using namespace r2l::gated;
using r2l::bf16;

namespace {

// Blocks of 8 warps where sequences are long: 128 positions of 32 channels a
// round (64 of 64 with 8-bit copies, whose scales span 64 channels), four
// groups of 8 rows per scheduler at 128 registers.  Blocks of 4 warps on 32
// positions of 64 channels where sequences are short, or middling and there
// are more than one wave of blocks: less of a block's life is its first tile.
// Measured, 4 and 8 warps: 8 x 4096 x 4096 channels 204 and 183 us, 8 x 128 x
// 4096 11 and 16 us, 256 ragged sequences of up to 512 389 and 632 us.
// Clusters of 2 do not pay here, the barrier undoes what a second block brings,
// except in ragged batches of odd rows, whose copies take longer (5 ragged x 777 x
// 515, fp32: single 20.1 us, clusters of 2 18.8; all of full length 21.3 and 34.7).
// fp32 rows are nearer to what memory gives, so fewer clusters of 4 pay (64 blocks
// of 600 positions: single 9.4 us, clusters of 4 11.5), and with their 8-bit copies
// clusters of 8 leave shared memory for one block an SM (one sequence of 2048 x
// 2048, 32 blocks: 47.1 us, clusters of 4 31.5).
Split forward_split(int B, int E, int L, int mode, int size, bool lengths) {
  const long long jobs64 = (long long)B * ((E - 1) / 64 + 1), jobs32 = (long long)B * ((E - 1) / 32 + 1);
  if (L < 512 || (L < 1024 && jobs64 > 592)) return {1, 4};
  if (mode == 2) return {cluster_of(jobs64, 64, L, {size == 2 ? 256 : 96, 256, 0}), 8};
  return {cluster_of(jobs32, 128, L, {256, size == 2 ? 256 : 192, lengths && E % (16 / size) ? 190 : 0}), 8};
}

// Whether every thread walks a sequence by itself: steps of one or two
// positions (2 positions of 8 x 1024 channels 3.1 us, in tiles 3.7; 4 positions
// 4.4 and 3.5), and short pieces of so many channels that tiles, filled by 8
// positions to a quarter, would take several waves (8192 rows of 4096 channels in
// pieces of 4 positions 117 us, in tiles 618; of 12 112 and 218, of 16 116 and
// 142, of 24 126 and 103).
bool walks(int B, int E, int L) {
  return L <= 2 || (L <= 16 && (long long)B * ((E - 1) / 64 + 1) > 592);
}

template <typename T, bool VEC, int MODE, int LANES, int WARPS>
r2l_status launch_shape(const FwdArgs& p, uint32_t blocks, cudaStream_t st) {
  using namespace r2l::gated;
  const long long jobs = (long long)p.B * ((p.E - 1) / (2 * LANES) + 1);
  return launch(gated_scan_kernel<T, VEC, MODE, LANES, WARPS>, p, jobs, blocks, WARPS * 32,
                fwd_smem_bytes<T, WHOLE_PIECES<T, VEC, MODE, WARPS>, LANES, WARPS>(blocks), st);
}
template <typename T, bool VEC, int MODE>
r2l_status launch_forward(const FwdArgs& p, Split c, cudaStream_t st) {
  if (c.warps == 4) return launch_shape<T, VEC, MODE, 32, 4>(p, c.blocks, st);
  return launch_shape<T, VEC, MODE, MODE == 2 ? 32 : 16, 8>(p, c.blocks, st);
}

template <typename T, bool VEC>
r2l_status run_forward(const FwdArgs& p, int mode, cudaStream_t st) {
  using namespace r2l::gated;
  if (mode == 0 && walks(p.B, p.E, p.L)) {
    const int pairs = (p.E + 1) / 2, threads = pairs <= 32 ? 32 : pairs <= 64 ? 64 : 128;
    const uint32_t blocks = (uint32_t)((pairs - 1) / threads + 1);
    const long long grid = (long long)p.B * blocks;
    if (grid > 2147483647LL) return R2L_ERR_UNSUPPORTED;
    gated_walk_kernel<T, VEC><<<(unsigned)grid, threads, 0, st>>>(p, blocks);
    R2L_LAUNCH_CHECK();
    return R2L_OK;
  }
  const Split c = forward_split(p.B, p.E, p.L, mode, sizeof(T), p.lengths != nullptr);
  if (mode == 0) return launch_forward<T, VEC, 0>(p, c, st);
  return mode == 1 ? launch_forward<T, VEC, 1>(p, c, st) : launch_forward<T, VEC, 2>(p, c, st);
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
  p.B = B; p.L = L; p.E = E; p.strips = (E - 1) / STRIP + 1;
  p.forward = (dims->flags & R2L_FLAG_FORWARD_SCAN) ? 1 : 0;
  p.lengths = lengths; p.status = status;
  if (train) {
    const CkptPlan k = plan_checkpoint(dims, B, L);
    if (!checkpoint || checkpoint_bytes < k.total) return R2L_ERR_WORKSPACE;
    if (!aligned(checkpoint, 16)) return R2L_ERR_ALIGNMENT;
    p.ck = checkpoint_at(k, checkpoint);
  }
  const int mode = !train ? 0 : (dims->flags & R2L_FLAG_ACT8) ? 2 : 1;
  const bool vec = E * es % 16 == 0 && rows16(p.x, p.ldx, es) && rows16(p.r, p.ldr, es) && rows16(p.g, p.ldg, es) &&
                   rows16(p.y, p.ldy, es);
  cudaStream_t st = (cudaStream_t)stream;
  if (dims->dtype == R2L_BF16) return vec ? run_forward<bf16, true>(p, mode, st) : run_forward<bf16, false>(p, mode, st);
  return vec ? run_forward<float, true>(p, mode, st) : run_forward<float, false>(p, mode, st);
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

}  // extern "C"
