// Kernels of the gated linear recurrence and of its gradient.
//
// In scan order k = 0, 1, …, per channel (rate = −R2L_GATED_RATE · softplus(lam)):
//
//   log a_k = rate · σ(r_k),  β_k = sqrt(1 − a_k²),  h_k = a_k h_{k−1} + β_k σ(g_k) x_k
//   G_k = dy_k + D_k,  D_{k−1} = a_k G_k   (D after the last position: dh_last)
//
// Both recurrences are affine maps of one number per channel, so a run of
// positions is one pair (A, B): out = A · in + B.  A block owns 64 channels of
// a sequence and takes 64 positions (a tile) at a time: every warp turns its
// share of the rows into a pair, the pairs of the warps before it give the
// value that enters the warp, and each row's result follows from it.  The rows
// of the next tile are on their way to shared memory meanwhile.  Where there
// are too few channels to fill the SMs, up to 8 blocks of a cluster take 8
// consecutive tiles at once and swap their tiles' pairs through distributed
// shared memory, one cluster barrier per 8 tiles: inputs are read once,
// whatever the split.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "act8.cuh"
#include "common.cuh"
#include "r2l.h"

namespace r2l {
namespace gated {

constexpr int TILE = R2L_GATED_TILE;     // positions per tile, and between two states of a checkpoint
constexpr int STRIP = R2L_ACT8_GROUP;    // channels per block: two per lane, and one scale of an 8-bit checkpoint
constexpr int MAX_CLUSTER = 8;           // the portable limit
constexpr int WALK_MAX = 8;              // positions up to which a thread walks a sequence by itself
static_assert(STRIP == 64, "a lane holds two channels");

// A checkpoint: states [B][tiles][strips·64] fp32 and, in 8 bits, x, r and g
// as [B][strips][L][64] bytes with scales [B][strips][Lp], rows in scan order:
// a tile's rows are contiguous for the one block that writes and reads them.
struct Ckpt {
  float* states;
  uint8_t* q[3];
  uint8_t* scales[3];
  int tiles, Lp;
};

struct FwdArgs {
  const void *x, *r, *g;
  long long ldx, ldr, ldg, ldy;
  const float *lam, *h0;
  void* y;
  float* h_last;
  int B, L, E, strips, forward;
  const int32_t* lengths;
  uint32_t* status;
  Ckpt ck;
};

struct BwdArgs {
  const void *x, *r, *g, *dy;
  long long ldx, ldr, ldg, ld_dy, ld_dx, ld_dr, ld_dg;
  const float *lam, *dh_last;
  void *dx, *dr, *dg;
  float *dh0, *part;      // part: [B · cluster][strips·64] partial sums of dlam
  int B, L, E, strips, forward;
  const int32_t* lengths;
  uint32_t* status;
  Ckpt ck;
};

// ---------------------------------------------------------------- arithmetic

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }

// −R2L_GATED_RATE · softplus(lam): log a at an open gate.
__device__ __forceinline__ float decay_rate(float lam) {
  return -R2L_GATED_RATE * (fmaxf(lam, 0.0f) + log1pf(expf(-fabsf(lam))));
}

// 1 / (1 + 2^(−v log2 e)): 0 at −∞ and 1 at +∞.
__device__ __forceinline__ float2 sigmoid2(float2 v) {
  const float2 t = __fmul2_rn(v, two(-LOG2E));
  const float2 d = __fadd2_rn(make_float2(ex2(t.x), ex2(t.y)), two(1.0f));
  return make_float2(rcp(d.x), rcp(d.y));
}

// The two channels of a lane at one position.  u = 1 − a² = −expm1(2 log a):
// above 2 log a = −1/4 the subtraction would lose the digits that matter (a
// channel with a memory of 1000 positions has 1 − a² = 0.002), so the Taylor
// polynomial of degree 6 is taken there (relative error under 5e-8).
struct Gates {
  float2 a, u, sr, sg;
};
__device__ __forceinline__ Gates gates2(float2 r, float2 g, float2 rate2 /* rate · log2 e */) {
  Gates q;
  q.sr = sigmoid2(r);
  q.sg = sigmoid2(g);
  const float2 l2 = __fmul2_rn(q.sr, rate2);
  q.a = make_float2(ex2(l2.x), ex2(l2.y));
  const float2 t = __fmul2_rn(l2, two(2.0f * LN2));
  const float2 far = __ffma2_rn(make_float2(-q.a.x, -q.a.y), q.a, two(1.0f));
  float2 c = __ffma2_rn(t, two(-1.0f / 720.0f), two(-1.0f / 120.0f));
  c = __ffma2_rn(c, t, two(-1.0f / 24.0f));
  c = __ffma2_rn(c, t, two(-1.0f / 6.0f));
  c = __ffma2_rn(c, t, two(-0.5f));
  c = __ffma2_rn(c, t, two(-1.0f));
  c = __fmul2_rn(c, t);
  q.u = make_float2(t.x > -0.25f ? c.x : far.x, t.y > -0.25f ? c.y : far.y);
  return q;
}

// ---------------------------------------------------------------- data movement

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

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 16 bytes to shared memory, the first `bytes` of them from src (the rest are zeros).
__device__ __forceinline__ void copy16(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

template <typename T>
__device__ __forceinline__ uint32_t bits_twice(float v);
template <>
__device__ __forceinline__ uint32_t bits_twice<float>(float v) {
  return __float_as_uint(v);
}
template <>
__device__ __forceinline__ uint32_t bits_twice<bf16>(float v) {
  return (__float_as_uint(v) >> 16) * 0x10001u;
}

// A tile of rows into dst[TILE][STRIP]: row k from src + k · step, its first
// `cols` channels; rows from `rows` on are filled with `fill` (bf16 holds it).
// VEC: every row starts on a 16-byte boundary.
template <typename T, bool VEC, int THREADS>
__device__ __forceinline__ void load_tile(T* dst, const T* src, long long step, int rows, int cols, float fill) {
  if (VEC) {
    constexpr int PER = 16 / (int)sizeof(T), CHUNKS = STRIP / PER;
#pragma unroll
    for (int i = 0; i < TILE * CHUNKS / THREADS; ++i) {
      const int row = (threadIdx.x + i * THREADS) / CHUNKS, c = (threadIdx.x + i * THREADS) % CHUNKS * PER;
      T* at = dst + row * STRIP + c;
      if (row < rows) {
        const int bytes = min(max(cols - c, 0), PER) * (int)sizeof(T);
        copy16(at, bytes ? src + row * step + c : src, bytes);
      } else {
        const uint32_t f = bits_twice<T>(fill);
        *reinterpret_cast<uint4*>(at) = make_uint4(f, f, f, f);
      }
    }
  } else {
    for (int i = threadIdx.x; i < TILE * STRIP; i += THREADS) {
      const int row = i / STRIP, c = i % STRIP;
      dst[i] = row < rows && c < cols ? src[row * step + c] : from_f32<T>(row < rows ? 0.0f : fill);
    }
  }
}

__device__ __forceinline__ float2 lane_pair(const float* row, int lane) {
  return reinterpret_cast<const float2*>(row)[lane];
}
__device__ __forceinline__ float2 lane_pair(const bf16* row, int lane) {
  const uint32_t v = reinterpret_cast<const uint32_t*>(row)[lane];
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// Channels 2·lane and 2·lane + 1 of a row of `cols` channels.  VEC: the pair is aligned.
template <bool VEC, typename T>
__device__ __forceinline__ float2 load_pair(const T* row, int lane, int cols) {
  if (VEC && 2 * lane + 1 < cols) return lane_pair(row, lane);
  return make_float2(2 * lane < cols ? to_f32(row[2 * lane]) : 0.0f, 2 * lane + 1 < cols ? to_f32(row[2 * lane + 1]) : 0.0f);
}
template <bool VEC>
__device__ __forceinline__ void store_pair(float* row, int lane, int cols, float2 v) {
  if (VEC && 2 * lane + 1 < cols) {
    reinterpret_cast<float2*>(row)[lane] = v;
  } else {
    if (2 * lane < cols) row[2 * lane] = v.x;
    if (2 * lane + 1 < cols) row[2 * lane + 1] = v.y;
  }
}
template <bool VEC>
__device__ __forceinline__ void store_pair(bf16* row, int lane, int cols, float2 v) {
  const __nv_bfloat162 w = __float22bfloat162_rn(v);
  if (VEC && 2 * lane + 1 < cols) {
    reinterpret_cast<__nv_bfloat162*>(row)[lane] = w;
  } else {
    if (2 * lane < cols) row[2 * lane] = w.x;
    if (2 * lane + 1 < cols) row[2 * lane + 1] = w.y;
  }
}
__device__ __forceinline__ float2 load_vec_pair(const float* v, int lane, int cols) {
  return make_float2(2 * lane < cols ? v[2 * lane] : 0.0f, 2 * lane + 1 < cols ? v[2 * lane + 1] : 0.0f);
}

// ---------------------------------------------------------------- clusters

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 16 bytes into the same shared variable of block `rank` of the cluster.
__device__ __forceinline__ void store_to_rank(const void* at, uint32_t rank, float4 v) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(at)), "r"(rank));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

// An affine map of a lane's two channels, (A.x, A.y, B.x, B.y), applied to v.
__device__ __forceinline__ float2 apply(float4 m, float2 v) {
  return __ffma2_rn(make_float2(m.x, m.y), v, make_float2(m.z, m.w));
}
// `second` after `first`.
__device__ __forceinline__ float4 after(float4 second, float4 first) {
  const float2 a = __fmul2_rn(make_float2(second.x, second.y), make_float2(first.x, first.y));
  const float2 b = apply(second, make_float2(first.z, first.w));
  return make_float4(a.x, a.y, b.x, b.y);
}

// The tiles' maps of one round through the cluster: `mine` is this block's, and
// `carry` the value that enters the first block's tile; returns the value that
// enters this block's and moves carry past the last block's.  box holds
// [blocks][32] maps and alternates between two buffers from round to
// round: a block writes a buffer again only after the barrier of the round
// between, which every reader of the buffer has passed.
__device__ __forceinline__ float2 through_cluster(float4* box, float4 mine, int warp, int warps, int lane, uint32_t rank,
                                                  uint32_t blocks, float2& carry) {
  for (uint32_t to = warp; to < blocks; to += warps) store_to_rank(box + rank * 32 + lane, to, mine);
  cluster_sync();
  float2 enters = carry;
  for (uint32_t q = 0; q < blocks; ++q) {
    if (q == rank) enters = carry;
    carry = apply(box[q * 32 + lane], carry);
  }
  return enters;
}

// ---------------------------------------------------------------- forward

constexpr int FW = 4;              // warps of a forward block
constexpr int FP = TILE / FW;      // rows of a warp

template <typename T>
struct FwdSmem {
  T in[2][3][TILE * STRIP];
  float4 maps[FW][32];
};
// The cluster's maps lie behind it: [2][blocks][32].
constexpr size_t box_bytes(uint32_t blocks) { return blocks > 1 ? 2 * (size_t)blocks * 32 * sizeof(float4) : 0; }

// MODE 0: the recurrence; 1: also the states of a checkpoint; 2: and its 8 bits.
template <typename T, bool VEC, int MODE>
__global__ void __launch_bounds__(FW * 32, sizeof(T) == 2 ? 4 : 2) gated_scan_kernel(const FwdArgs p, const uint32_t blocks) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  FwdSmem<T>& sm = *reinterpret_cast<FwdSmem<T>*>(smem_raw);
  float4* const box = reinterpret_cast<float4*>(smem_raw + sizeof(FwdSmem<T>));
  if (p.status && blockIdx.x == 0) write_status(p.lengths, p.B, p.L, p.status);
  const uint32_t rank = blockIdx.x % blocks;
  const uint32_t job = blockIdx.x / blocks;
  const int strip = (int)(job % (uint32_t)p.strips), b = (int)(job / (uint32_t)p.strips);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e0 = strip * STRIP, cols = min(p.E - e0, STRIP);
  const int n = clamped_length(p.lengths, b, p.L);
  const long long row0 = (long long)b * p.L + (p.forward ? 0 : n - 1);   // row of position k: row0 ± k
  const int dir = p.forward ? 1 : -1;
  const float2 lam = load_vec_pair(p.lam + e0, lane, cols);
  const float2 rate2 = make_float2(decay_rate(lam.x) * LOG2E, decay_rate(lam.y) * LOG2E);
  float2 carry = p.h0 ? load_vec_pair(p.h0 + (size_t)b * p.E + e0, lane, cols) : two(0.0f);

  const T* const src[3] = {(const T*)p.x + row0 * p.ldx + e0, (const T*)p.r + row0 * p.ldr + e0,
                           (const T*)p.g + row0 * p.ldg + e0};
  const long long step[3] = {dir * p.ldx, dir * p.ldr, dir * p.ldg};
  // A position past the end has r = −∞ and x = 0: a = 1, b = 0, and no other
  // test is needed in the arithmetic.
  auto load = [&](int round) {
    const long long k0 = ((long long)round * blocks + rank) * TILE;
    if (k0 < n)
#pragma unroll
      for (int i = 0; i < 3; ++i)
        load_tile<T, VEC, FW * 32>(sm.in[round & 1][i], src[i] + k0 * step[i], step[i], (int)min((long long)TILE, n - k0),
                                   cols, i == 1 ? -INFINITY : 0.0f);
    copies_commit();
  };

  const int rounds = (int)(((long long)n + TILE * blocks - 1) / (TILE * blocks));
  if (rounds > 0) load(0);
  if (rounds > 1) load(1);
  else copies_commit();
  if (blocks > 1) cluster_sync();   // every block of the cluster runs before its shared memory is written
  for (int round = 0; round < rounds; ++round) {
    const int buf = round & 1;
    const long long k0 = ((long long)round * blocks + rank) * TILE;
    const int rows = (int)max(0ll, min((long long)TILE, n - k0));   // of this block's tile
    copies_wait<1>();
    __syncthreads();
    float2 P[FP], H[FP];     // row j's state is P[j] · (state that enters the warp) + H[j]
    float2 a = two(1.0f), h = two(0.0f);
    const int mine = rows - warp * FP;   // rows of this warp
    if (mine > 0) {
#pragma unroll
      for (int j = 0; j < FP; ++j) {
        const int at = (warp * FP + j) * STRIP;
        const float2 x = lane_pair(sm.in[buf][0] + at, lane), r = lane_pair(sm.in[buf][1] + at, lane),
                     g = lane_pair(sm.in[buf][2] + at, lane);
        const Gates q = gates2(r, g, rate2);
        const float2 bx = __fmul2_rn(make_float2(sqrt_approx(q.u.x), sqrt_approx(q.u.y)), __fmul2_rn(q.sg, x));
        a = __fmul2_rn(a, q.a);
        h = __ffma2_rn(q.a, h, bx);
        P[j] = a;
        H[j] = h;
      }
    }
    sm.maps[warp][lane] = make_float4(a.x, a.y, h.x, h.y);
    if (MODE == 2 && mine > 0) {
      // The group of 64 channels that shares a scale is one row of the warp.
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const size_t tile = ((size_t)b * p.strips + strip) * p.L + k0 + warp * FP;
        uint32_t keep = 0;
#pragma unroll
        for (int j = 0; j < FP; ++j) {
          const float2 v = lane_pair(sm.in[buf][i] + (warp * FP + j) * STRIP, lane);
          const uint32_t top = __reduce_max_sync(0xffffffffu, max(act8::finite_abs_bits(v.x), act8::finite_abs_bits(v.y)));
          const uint32_t byte = act8::scale_byte(top);
          const float down = act8::scale_down(byte);
          if (lane == j) keep = byte;
          if (j < mine)
            reinterpret_cast<uint16_t*>(p.ck.q[i] + (tile + j) * STRIP)[lane] =
                act8::to_e4m3x2(act8::nan_if_not_finite(v.x) * down, act8::nan_if_not_finite(v.y) * down);
        }
        if (lane < FP && lane < mine)
          p.ck.scales[i][((size_t)b * p.strips + strip) * p.ck.Lp + k0 + warp * FP + lane] = (uint8_t)keep;
      }
    }
    __syncthreads();
    if (round + 2 < rounds) load(round + 2);
    else copies_commit();
    // the value that enters this tile, then this warp
    float2 enters;
    if (blocks > 1) {
      float4 tile = sm.maps[0][lane];
#pragma unroll
      for (int w = 1; w < FW; ++w) tile = after(sm.maps[w][lane], tile);
      enters = through_cluster(box + buf * blocks * 32, tile, warp, FW, lane, rank, blocks, carry);
    } else {
      enters = carry;
#pragma unroll
      for (int w = 0; w < FW; ++w) carry = apply(sm.maps[w][lane], carry);
    }
    if (MODE >= 1 && warp == 0 && rows > 0)
      reinterpret_cast<float2*>(p.ck.states + ((size_t)b * p.ck.tiles + k0 / TILE) * p.strips * STRIP + e0)[lane] = enters;
#pragma unroll
    for (int w = 0; w < FW - 1; ++w)
      if (w < warp) enters = apply(sm.maps[w][lane], enters);
    T* out = (T*)p.y + (row0 + dir * (k0 + warp * FP)) * p.ldy + e0;
#pragma unroll
    for (int j = 0; j < FP; ++j)
      if (j < mine) store_pair<VEC>(out + j * dir * p.ldy, lane, cols, __ffma2_rn(P[j], enters, H[j]));
  }
  if (p.h_last && rank == 0 && warp == 0) store_pair<false>(p.h_last + (size_t)b * p.E + e0, lane, cols, carry);
}

// A few positions (a step of decoding): a thread walks its two channels.
template <typename T, bool VEC>
__global__ void __launch_bounds__(128) gated_walk_kernel(const FwdArgs p) {
  if (p.status && blockIdx.x == 0) write_status(p.lengths, p.B, p.L, p.status);
  const int pairs = (p.E + 1) / 2;
  const long long at = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const int b = (int)(at / pairs), pair = (int)(at % pairs);
  if (b >= p.B) return;
  const int n = clamped_length(p.lengths, b, p.L);
  const float2 lam = load_vec_pair(p.lam, pair, p.E);
  const float2 rate2 = make_float2(decay_rate(lam.x) * LOG2E, decay_rate(lam.y) * LOG2E);
  float2 h = p.h0 ? load_vec_pair(p.h0 + (size_t)b * p.E, pair, p.E) : two(0.0f);
  for (int k = 0; k < n; ++k) {
    const long long m = (long long)b * p.L + (p.forward ? k : n - 1 - k);
    const Gates q = gates2(load_pair<VEC>((const T*)p.r + m * p.ldr, pair, p.E),
                           load_pair<VEC>((const T*)p.g + m * p.ldg, pair, p.E), rate2);
    const float2 x = load_pair<VEC>((const T*)p.x + m * p.ldx, pair, p.E);
    h = __ffma2_rn(q.a, h, __fmul2_rn(make_float2(sqrt_approx(q.u.x), sqrt_approx(q.u.y)), __fmul2_rn(q.sg, x)));
    store_pair<VEC>((T*)p.y + m * p.ldy, pair, p.E, h);
  }
  if (p.h_last) store_pair<false>(p.h_last + (size_t)b * p.E, pair, p.E, h);
}

}  // namespace gated
}  // namespace r2l
