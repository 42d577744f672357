// The gated linear recurrence (r2l_gated_scan, its training forward and its
// gradient) and the 8-bit activation checkpoints (r2l_act8_pack / _unpack):
// kernels, argument checks and launches.
#include <algorithm>
#include <cstdint>

#include "act8.cuh"
#include "common.cuh"
#include "r2l.h"

using r2l::bf16;
using r2l::from_f32;
using r2l::to_f32;

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

// ------------------------------------------------------------------ device

__device__ __forceinline__ int clamped_length(const int32_t* lengths, int b, int L) {
  return lengths ? min(max(lengths[b], 0), L) : L;
}

// One block writes the status word: whether any length lies outside [0, L].
__device__ __forceinline__ void write_status(const int32_t* lengths, int B, int L, uint32_t* status) {
  int bad = 0;
  if (lengths)
    for (int b = threadIdx.x; b < B; b += blockDim.x) bad |= lengths[b] < 0 || lengths[b] > L;
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) *status = bad ? R2L_DEVFLAG_LENGTH_CLAMPED : 0u;
}

__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

// −R2L_GATED_RATE · softplus(lam): the log of the decay at an open gate.
__device__ __forceinline__ float decay_rate(float lam) {
  return -R2L_GATED_RATE * (fmaxf(lam, 0.0f) + log1pf(expf(-fabsf(lam))));
}

struct Gates {
  float a, beta, sr, sg, l;
};
__device__ __forceinline__ Gates gates(float r, float g, float rate) {
  Gates q;
  q.sr = sigmoid(r);
  q.sg = sigmoid(g);
  q.l = rate * q.sr;
  q.a = expf(q.l);
  q.beta = sqrtf(-expm1f(2.0f * q.l));
  return q;
}

struct Ckpt {
  float* states;        // [B][tiles][E]
  uint8_t* q[3];        // x, r, g: [B·L][ldq]
  uint8_t* scales[3];   // [B·L][ldq / GROUP]
  int tiles, ldq;
};

struct FwdArgs {
  const void *x, *r, *g;
  long long ldx, ldr, ldg, ldy;
  const float *lam, *h0;
  void* y;
  float* h_last;
  int B, L, E, forward;
  const int32_t* lengths;
  uint32_t* status;
  Ckpt ck;
};

struct BwdArgs {
  const void *x, *r, *g, *dy;
  long long ldx, ldr, ldg, ld_dy, ld_dx, ld_dr, ld_dg;
  const float *lam, *dh_last;
  void *dx, *dr, *dg;
  float *dlam, *dh0, *part;
  int B, L, E, forward, act8;
  const int32_t* lengths;
  uint32_t* status;
  Ckpt ck;
};

template <typename T>
__global__ void gated_fwd_kernel(FwdArgs p) {
  if (p.status && blockIdx.x == 0 && blockIdx.y == 0) write_status(p.lengths, p.B, p.L, p.status);
  const int e = blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.y;
  if (e >= p.E) return;
  const int n = clamped_length(p.lengths, b, p.L);
  const float rate = decay_rate(p.lam[e]);
  float h = p.h0 ? p.h0[(size_t)b * p.E + e] : 0.0f;
  for (int k = 0; k < n; ++k) {
    if (p.ck.states && k % TILE == 0) p.ck.states[((size_t)b * p.ck.tiles + k / TILE) * p.E + e] = h;
    const long long m = (long long)b * p.L + (p.forward ? k : n - 1 - k);
    const Gates q = gates(to_f32(((const T*)p.r)[m * p.ldr + e]), to_f32(((const T*)p.g)[m * p.ldg + e]), rate);
    h = q.a * h + q.beta * q.sg * to_f32(((const T*)p.x)[m * p.ldx + e]);
    ((T*)p.y)[m * p.ldy + e] = from_f32<T>(h);
  }
  if (p.h_last) p.h_last[(size_t)b * p.E + e] = h;
}

template <typename T>
__device__ __forceinline__ float load_in(const BwdArgs& p, int which, const void* ptr, long long ld, long long m, int e) {
  if (!p.act8) return to_f32(((const T*)ptr)[m * ld + e]);
  const float up = r2l::act8::scale_up(p.ck.scales[which][m * (p.ck.ldq / GROUP) + e / GROUP]);
  return r2l::act8::from_e4m3x2(p.ck.q[which][m * p.ck.ldq + e]).x * up;
}

template <typename T>
__global__ void gated_bwd_kernel(BwdArgs p) {
  if (blockIdx.x == 0 && blockIdx.y == 0) write_status(p.lengths, p.B, p.L, p.status);
  const int e = blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.y;
  if (e >= p.E) return;
  const int n = clamped_length(p.lengths, b, p.L);
  const float rate = decay_rate(p.lam[e]);
  float D = p.dh_last ? p.dh_last[(size_t)b * p.E + e] : 0.0f, acc = 0.0f;
  float enters[TILE];
  for (int t = (n + TILE - 1) / TILE - 1; t >= 0; --t) {
    float h = p.ck.states[((size_t)b * p.ck.tiles + t) * p.E + e];
    const int k0 = t * TILE, k1 = min(n, k0 + TILE);
    for (int k = k0; k < k1; ++k) {
      const long long m = (long long)b * p.L + (p.forward ? k : n - 1 - k);
      enters[k - k0] = h;
      const Gates q = gates(load_in<T>(p, 1, p.r, p.ldr, m, e), load_in<T>(p, 2, p.g, p.ldg, m, e), rate);
      h = q.a * h + q.beta * q.sg * load_in<T>(p, 0, p.x, p.ldx, m, e);
    }
    for (int k = k1 - 1; k >= k0; --k) {
      const long long m = (long long)b * p.L + (p.forward ? k : n - 1 - k);
      const float x = load_in<T>(p, 0, p.x, p.ldx, m, e);
      const Gates q = gates(load_in<T>(p, 1, p.r, p.ldr, m, e), load_in<T>(p, 2, p.g, p.ldg, m, e), rate);
      const float G = D + to_f32(((const T*)p.dy)[m * p.ld_dy + e]);
      const float dl = q.l == 0.0f ? 0.0f : G * (q.a * enters[k - k0] - q.sg * x * q.a * q.a / q.beta);
      ((T*)p.dx)[m * p.ld_dx + e] = from_f32<T>(G * q.beta * q.sg);
      ((T*)p.dg)[m * p.ld_dg + e] = from_f32<T>(G * q.beta * x * q.sg * (1.0f - q.sg));
      ((T*)p.dr)[m * p.ld_dr + e] = from_f32<T>(dl * q.l * (1.0f - q.sr));
      acc += dl * q.sr;
      D = G * q.a;
    }
  }
  for (int i = n; i < p.L; ++i) {
    const long long m = (long long)b * p.L + i;
    ((T*)p.dx)[m * p.ld_dx + e] = ((T*)p.dg)[m * p.ld_dg + e] = ((T*)p.dr)[m * p.ld_dr + e] = from_f32<T>(0.0f);
  }
  p.part[(size_t)b * p.E + e] = acc;
  if (p.dh0) p.dh0[(size_t)b * p.E + e] = D;
}

__global__ void gated_dlam_kernel(const float* part, int rows, const float* lam, int E, float* dlam) {
  const int e = blockIdx.x * blockDim.x + threadIdx.x;
  if (e >= E) return;
  float s = 0.0f;
  for (int i = 0; i < rows; ++i) s += part[(size_t)i * E + e];
  dlam[e] = s * -R2L_GATED_RATE * sigmoid(lam[e]);
}

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
  int tiles, ldq;
};
CkptPlan plan_checkpoint(const r2l_dims* d, int B, int L) {
  CkptPlan k{};
  const size_t M = (size_t)B * L, E = d->d_inner;
  k.tiles = (L - 1) / TILE + 1;
  k.ldq = (int)align_up(E, GROUP);
  size_t off = 0;
  k.states = off;
  off = align_up(off + (size_t)B * k.tiles * E * sizeof(float), kAlign);
  if (d->flags & R2L_FLAG_ACT8)
    for (int i = 0; i < 3; ++i) {
      k.q[i] = off;
      off = align_up(off + M * k.ldq, kAlign);
      k.scales[i] = off;
      off = align_up(off + M * (k.ldq / GROUP), kAlign);
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
  ck.ldq = k.ldq;
  return ck;
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
  if (!fits(B, L, E) || B > 65535) return R2L_ERR_UNSUPPORTED;
  FwdArgs p{};
  p.x = in->x; p.r = in->r; p.g = in->g;
  p.ldx = in->ldx; p.ldr = in->ldr; p.ldg = in->ldg; p.ldy = ldy;
  p.lam = in->lam; p.h0 = in->h0; p.y = y; p.h_last = h_last;
  p.B = B; p.L = L; p.E = E; p.forward = (dims->flags & R2L_FLAG_FORWARD_SCAN) ? 1 : 0;
  p.lengths = lengths; p.status = status;
  cudaStream_t st = (cudaStream_t)stream;
  if (train) {
    const CkptPlan k = plan_checkpoint(dims, B, L);
    if (!checkpoint || checkpoint_bytes < k.total) return R2L_ERR_WORKSPACE;
    if (!aligned(checkpoint, 16)) return R2L_ERR_ALIGNMENT;
    p.ck = checkpoint_at(k, checkpoint);
  }
  if (train && (dims->flags & R2L_FLAG_ACT8)) {
    const void* src[3] = {in->x, in->r, in->g};
    const int ld[3] = {in->ldx, in->ldr, in->ldg};
    for (int i = 0; i < 3; ++i)
      R2L_TRY(act8_pack(src[i], ld[i], dims->dtype, B, L, E, lengths, p.ck.q[i], p.ck.ldq, p.ck.scales[i], st));
  }
  const dim3 grid((E + 63) / 64, B);
  if (dims->dtype == R2L_BF16) gated_fwd_kernel<bf16><<<grid, 64, 0, st>>>(p);
  else gated_fwd_kernel<float><<<grid, 64, 0, st>>>(p);
  R2L_LAUNCH_CHECK();
  return R2L_OK;
}

size_t part_bytes(const r2l_dims* d, int B) { return (size_t)B * d->d_inner * sizeof(float); }

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
  return valid_dims(dims, B, L) && fits(B, L, dims->d_inner) ? kAlign + align_up(part_bytes(dims, B), kAlign) : 0;
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
  if (!fits(B, L, E) || B > 65535) return R2L_ERR_UNSUPPORTED;
  const CkptPlan k = plan_checkpoint(dims, B, L);
  if (!checkpoint || checkpoint_bytes < k.total) return R2L_ERR_WORKSPACE;
  if (!workspace || workspace_bytes < r2l_gated_scan_backward_workspace_size(dims, B, L)) return R2L_ERR_WORKSPACE;
  if (!aligned(checkpoint, 16) || !aligned(workspace, 16)) return R2L_ERR_ALIGNMENT;
  BwdArgs p{};
  p.x = in->x; p.r = in->r; p.g = in->g; p.dy = dy;
  p.ldx = in->ldx; p.ldr = in->ldr; p.ldg = in->ldg; p.ld_dy = ld_dy;
  p.dx = grads->dx; p.dr = grads->dr; p.dg = grads->dg;
  p.ld_dx = grads->ld_dx; p.ld_dr = grads->ld_dr; p.ld_dg = grads->ld_dg;
  p.lam = in->lam; p.dh_last = dh_last; p.dlam = grads->dlam; p.dh0 = grads->dh0;
  p.part = (float*)((char*)workspace + kAlign);
  p.B = B; p.L = L; p.E = E; p.forward = (dims->flags & R2L_FLAG_FORWARD_SCAN) ? 1 : 0; p.act8 = act8;
  p.lengths = lengths; p.status = (uint32_t*)workspace;
  p.ck = checkpoint_at(k, const_cast<void*>(checkpoint));
  cudaStream_t st = (cudaStream_t)stream;
  const dim3 grid((E + 63) / 64, B);
  if (dims->dtype == R2L_BF16) gated_bwd_kernel<bf16><<<grid, 64, 0, st>>>(p);
  else gated_bwd_kernel<float><<<grid, 64, 0, st>>>(p);
  R2L_LAUNCH_CHECK();
  gated_dlam_kernel<<<(E + 127) / 128, 128, 0, st>>>(p.part, B, p.lam, E, p.dlam);
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
