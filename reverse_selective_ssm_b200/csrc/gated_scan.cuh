// Kernels of the gated linear recurrence and of its gradient.
//
// In scan order k = 0, 1, …, per channel (rate = −R2L_GATED_RATE · softplus(lam)):
//
//   log a_k = rate · σ(r_k),  β_k = sqrt(1 − a_k²),  h_k = a_k h_{k−1} + β_k σ(g_k) x_k
//   G_k = dy_k + D_k,  D_{k−1} = a_k G_k   (D after the last position: dh_last)
//
// Both recurrences are affine maps of one number per channel, so a run of
// positions is one pair (A, B): out = A · in + B.  A block owns 32 or 64
// channels of a sequence.  Its warps take 8 or 16 consecutive positions each;
// a warp turns its rows into one pair while it waits for nothing, then gets the
// state that enters from the warp before, hands on the one that leaves and
// writes its rows.  The rows of the warp's next two turns are on their way to
// shared memory meanwhile.  Where there are too few channels to fill the SMs,
// up to 8 blocks of a cluster take consecutive tiles at once and swap their
// tiles' pairs through distributed shared memory, one cluster barrier a round:
// inputs are read once, whatever the split.
//
// What bounds it (B200, bf16, 8 sequences of 4096 positions, 4096 channels):
// 8 bytes per position and channel, 164 us at the measured copy rate, against
// 34 instructions (of which 4 are special functions) per 32 of them.  The scan
// takes 183 us (5.9 TB/s); under a sustained load that brings the SM clock down
// to 1.57 GHz, 220 us.  In fp32 (8 x 2048 x 4096) it takes 168 us, 6.4 TB/s.
// 16 warps an SM at 128 registers beat 28 at 72 (184 and 194 us): the eight
// rows of a thread overlap each other's special functions.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "act8.cuh"
#include "common.cuh"
#include "r2l.h"

namespace r2l {
namespace gated {

constexpr int TILE = R2L_GATED_TILE;     // positions per tile, and between two states of a checkpoint
constexpr int STRIP = R2L_ACT8_GROUP;    // channels that share a scale of an 8-bit checkpoint
constexpr int MAX_CLUSTER = 8;           // the portable limit
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
constexpr float LOG2E_REST = (float)(1.4426950408889634 - (double)LOG2E);     // log2 e − LOG2E

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

// −R2L_GATED_RATE · softplus(lam), log a at an open gate.  With e = e^−|lam|
// (the rounding of the exponent's product made up for) and z = e / (2 + e),
// log(1 + e) = 2 atanh z = 2z (1 + z²/3 + z⁴/5 + …), z ≤ 1/3: seven terms leave
// a relative error of a few 2^-24, in a fifth of the instructions of
// log1pf(expf()), which were most of a decoding step.  An e below 2^-126
// (lam < −87) counts as 0, a decay that fp32 cannot tell from 1; |lam| is held to
// 128 there, so that ±∞ makes no ∞ − ∞.  softplus(lam) is held to 2^124: log2 a
// at an open gate is then finite, and 0 times it, a closed gate, is 0 for every
// lam.  A NaN passes both limits.
constexpr float SOFTPLUS_MAX = 0x1p124f;
__device__ __forceinline__ float decay_rate(float lam) {
  const float w = -fabsf(lam), v = w < -128.0f ? -128.0f : w, t = v * LOG2E;
  const float rest = fmaf(v, LOG2E, -t) + v * LOG2E_REST;     // of v · log2 e
  const float e0 = ex2(t), e = fmaf(e0, rest * LN2, e0);
  const float z = e * rcp(2.0f + e), q = z * z;
  float c = fmaf(q, 1.0f / 15.0f, 1.0f / 13.0f);
  c = fmaf(c, q, 1.0f / 11.0f);
  c = fmaf(c, q, 1.0f / 9.0f);
  c = fmaf(c, q, 1.0f / 7.0f);
  c = fmaf(c, q, 1.0f / 5.0f);
  c = fmaf(c, q, 1.0f / 3.0f);
  c = fmaf(c, q, 1.0f);
  return -R2L_GATED_RATE * fmaf(2.0f * z, c, fminf(fmaxf(lam, 0.0f), SOFTPLUS_MAX));
}

// 1 + 2^(−v log2 e), whose reciprocal is σ(v): ∞ at −∞ and 1 at +∞.
__device__ __forceinline__ float2 sigmoid_den(float2 v) {
  const float2 t = __fmul2_rn(v, two(-LOG2E));
  return __fadd2_rn(make_float2(ex2(t.x), ex2(t.y)), two(1.0f));
}
__device__ __forceinline__ float2 sigmoid2(float2 v) {
  const float2 d = sigmoid_den(v);
  return make_float2(rcp(d.x), rcp(d.y));
}

// Any decay: u = 1 − a² = −expm1(2 log a).  Where a is near 1 the subtraction
// would lose the digits that matter (a channel with a memory of 1000 positions
// has 1 − a² = 0.002), so for log2 a above −0.18 it is a polynomial in log2 a
// without a constant term, fitted for the least relative error (4 · 2^-24).
struct Gates {
  float2 a, u, sr, sg;
};
__device__ __forceinline__ Gates gates2(float2 r, float2 g, float2 rate2 /* rate · log2 e */) {
  Gates q;
  q.sr = sigmoid2(r);
  q.sg = sigmoid2(g);
  const float2 l2 = __fmul2_rn(q.sr, rate2);
  q.a = make_float2(ex2(l2.x), ex2(l2.y));
  const float2 far = __ffma2_rn(__fmul2_rn(q.a, q.a), two(-1.0f), two(1.0f));
  float2 c = __ffma2_rn(l2, two(-0.139302522f), two(-0.442409396f));
  c = __ffma2_rn(c, l2, two(-0.960847378f));
  c = __ffma2_rn(c, l2, two(-1.38629401f));
  c = __fmul2_rn(c, l2);
  q.u = make_float2(l2.x > -0.18f ? c.x : far.x, l2.y > -0.18f ? c.y : far.y);
  return q;
}

// Channels that keep at least 0.71 of their state per position at an open gate
// (−0.5 ≤ rate2 ≤ 0; a recurrence with a memory of a few positions or more).
// With s = 1/√(1 + e^−r), σ(r) = s² and β = s · k · p(log2 a), where
// k = √(−2 ln 2 · rate2) and p is smooth: one reciprocal square root gives the
// gate and β's square root, and a is a polynomial too, so a position takes four
// special-function operations instead of six, and no choice by cases.  Both
// polynomials are fitted on [−0.5, 0] for the least relative error (under 2^-24).
// 8 x 4096 x 4096, bf16: scan 185 us, gradient 396; with any decay (above) 219
// and 449.  A block decides by its channels' lam.
constexpr float NEAR_RATE2 = -0.5f;
__device__ __forceinline__ float2 near_decay(float2 l2) {   // 2^l2
  float2 c = __ffma2_rn(l2, two(0.00115445221f), two(0.0095412815f));
  c = __ffma2_rn(c, l2, two(0.0554904081f));
  c = __ffma2_rn(c, l2, two(0.240225643f));
  c = __ffma2_rn(c, l2, two(0.693147182f));
  return __ffma2_rn(c, l2, two(1.0f));
}
__device__ __forceinline__ float2 near_beta(float2 l2) {    // √((1 − 2^(2 l2)) / (−2 ln 2 · l2))
  float2 c = __ffma2_rn(l2, two(0.00273338961f), two(0.0206286889f));
  c = __ffma2_rn(c, l2, two(0.100061379f));
  c = __ffma2_rn(c, l2, two(0.346571505f));
  return __ffma2_rn(c, l2, two(1.0f));
}
__device__ __forceinline__ float2 near_scale(float2 rate2) {   // k
  return make_float2(sqrtf(-2.0f * LN2 * rate2.x), sqrtf(-2.0f * LN2 * rate2.y));
}

// a and b = β σ(g) x at one position.
template <bool NEAR>
__device__ __forceinline__ void coefficients(float2 x, float2 r, float2 g, float2 rate2, float2 k, float2& a, float2& b) {
  if (NEAR) {
    const float2 d = sigmoid_den(r);
    const float2 s = make_float2(rsqrt_approx(d.x), rsqrt_approx(d.y));
    const float2 l2 = __fmul2_rn(__fmul2_rn(s, s), rate2);
    a = near_decay(l2);
    b = __fmul2_rn(__fmul2_rn(__fmul2_rn(s, k), near_beta(l2)), __fmul2_rn(sigmoid2(g), x));
  } else {
    const Gates q = gates2(r, g, rate2);
    a = q.a;
    b = __fmul2_rn(make_float2(sqrt_approx(q.u.x), sqrt_approx(q.u.y)), __fmul2_rn(q.sg, x));
  }
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

// 16 bytes to an address of shared memory; zeros where they do not exist (src is valid all the same).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool exists = true) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %2, 0;\n\tcp.async.cg.shared.global [%0], [%1], 16, p;\n\t}" ::"r"(dst),
               "l"(src), "r"((uint32_t)exists)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// Threads of a warp and their rows.  LANES lanes hold a row of 2 · LANES
// channels, two each, so a warp has 32 / LANES groups of ROWS consecutive rows;
// in shared memory a group is followed by 64 bytes of nothing, which puts two
// groups that are read together into different banks.  ANY: rows start
// anywhere in memory; a row in shared memory then starts as far from a
// 16-byte boundary as in memory, and has 16 bytes more.
template <typename T, int LANES, int ROWS, bool ANY>
struct Layout {
  static constexpr int CHANNELS = 2 * LANES;
  static constexpr int GROUPS = 32 / LANES;                  // of a warp
  static constexpr int PER = 16 / (int)sizeof(T);            // elements of a copy
  static constexpr int ROW = CHANNELS + (ANY ? PER : 0);     // elements from row to row
  static constexpr int GROUP_STRIDE = ROWS * ROW + (GROUPS > 1 && !ANY ? 64 / (int)sizeof(T) : 0);
  static constexpr int WARP_STRIDE = GROUPS * GROUP_STRIDE;
  static constexpr int CHUNKS = CHANNELS / PER;              // copies of a row
  static constexpr int AT_ONCE = 32 / CHUNKS;                // rows that a warp's lanes copy at once
  static constexpr int WARP_ROWS = ROWS * GROUPS;
  static_assert(ANY || ROWS % AT_ONCE == 0 || AT_ONCE == WARP_ROWS, "at(i + j) = at(i) + at(j) for the rows of a copy");
  static __device__ __forceinline__ int at(int row) { return row / ROWS * GROUP_STRIDE + row % ROWS * ROW; }
  // This lane's chunk of the first rows that are copied at once.
  static __device__ __forceinline__ int chunk(int wl) { return at(wl / CHUNKS) + channel(wl); }
  static __device__ __forceinline__ int channel(int wl) { return wl % CHUNKS * PER; }
};

// The rows of a warp from position k on, on their way to dst in shared memory.
// A warp copies only the rows that it reads itself, so a copy needs no barrier
// of the block.  `step` leads to the next position.  Rows past the last
// position n − 1 take that one's values (no test per copy; see fill_rows).
// copy_rows: rows start on 16-byte boundaries and channels come in multiples of
// them, so a chunk exists or does not; `first` is position 0 at this lane's
// channel() (any valid one if it does not exist), `dst` this lane's chunk of
// the warp's rows: an address is one multiply-add.
template <typename T, typename LAY>
__device__ __forceinline__ void copy_rows(uint32_t dst, const T* first, int step, int k, int n, int wl, bool exists) {
  k += wl / LAY::CHUNKS;
#pragma unroll
  for (int i = 0; i < LAY::WARP_ROWS; i += LAY::AT_ONCE)
    copy16(dst + LAY::at(i) * (int)sizeof(T), first + (long long)min(k + i, n - 1) * step, exists);
}

// Elements from the 16-byte boundary before position k (of a sequence whose
// position 0 is at `first`) to it.
template <typename T>
__device__ __forceinline__ int offset_of(const T* first, int step, int k) {
  return (int)((uint32_t)((uintptr_t)first / sizeof(T)) + (uint32_t)k * (uint32_t)step) & (16 / (int)sizeof(T) - 1);
}
// Positions of a sequence whose row has nothing of the array before it, or
// nothing behind it (−1: none).
struct Edges {
  int head, tail;
};
__device__ __forceinline__ Edges array_edges(int b, int B, int n, int L, bool forward) {
  return {b == 0 && n > 0 ? (forward ? 0 : n - 1) : -1, b == B - 1 && n == L ? (forward ? L - 1 : 0) : -1};
}
// copy_any: rows that start anywhere.  The 16-byte pieces of memory that hold
// a row's channels are copied whole, with what they hold of the rows beside
// it, which no result uses; the array's first and last row, whose pieces may
// reach outside it, go element by element, as do rows shorter than a piece.
// `first` is position 0 at the block's first channel, of which `cols` exist.
// All rows element by element: 61 ragged x 512 x 1037, fp32, 100 us, here 70;
// 8 x 2000 x 1037, bf16, 86 and 53.
template <typename T, typename LAY>
__device__ __forceinline__ void copy_any(T* dst, const T* first, int step, int k, int n, int cols, const Edges& edges, int wl) {
  constexpr int PIECES = LAY::CHUNKS + 1;
#pragma unroll
  for (int i = 0; i < (LAY::WARP_ROWS * PIECES + 31) / 32; ++i) {
    const int row = (i * 32 + wl) / PIECES, piece = (i * 32 + wl) % PIECES, pos = min(k + row, n - 1);
    const int from = piece * LAY::PER - offset_of(first, step, pos);      // channel at the piece's start
    if (row >= LAY::WARP_ROWS || from >= cols) continue;
    T* const to = dst + LAY::at(row) + piece * LAY::PER;
    const T* const src = first + (long long)pos * step + from;
    if (pos != edges.head && pos != edges.tail && abs(step) >= LAY::PER) {
      copy16(smem_addr(to), src);
    } else {
      for (int c = 0; c < LAY::PER; ++c)
        if (from + c >= 0 && from + c < cols) to[c] = src[c];
    }
  }
}
// One element to shared memory, or 0 where it does not exist (`from` is valid all the same).
__device__ __forceinline__ void copy_element(float* to, const float* from, bool exists) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(to)), "l"(from), "r"(exists ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copy_element(bf16* to, const bf16* from, bool exists) {
  *to = exists ? *from : from_f32<bf16>(0.0f);
}

// copy_elements: the same rows element by element, into rows of shared memory
// that start at their channel 0, with 0 in channels that do not exist.
template <typename T, typename LAY>
__device__ __forceinline__ void copy_elements(T* dst, const T* first, int step, int k, int n, int cols, int wl) {
  static_assert(LAY::CHANNELS % 32 == 0, "a lane copies a channel");
#pragma unroll
  for (int c = 0; c < LAY::CHANNELS; c += 32) {
    const bool exists = c + wl < cols;
    const T* const from = first + (exists ? c + wl : 0);
#pragma unroll 8
    for (int row = 0; row < LAY::WARP_ROWS; ++row)
      copy_element(dst + LAY::at(row) + c + wl, from + (long long)min(k + row, n - 1) * step, exists);
  }
}

// v in all channels of the rows from `rows` on, of a warp that has no more.
template <typename T, typename LAY>
__device__ __forceinline__ void fill_rows(T* dst, int wl, int rows, float v) {
#pragma unroll 1
  for (int row = rows; row < LAY::WARP_ROWS; ++row)
    for (int c = wl; c < LAY::ROW; c += 32) dst[LAY::at(row) + c] = from_f32<T>(v);
}

__device__ __forceinline__ float2 lane_pair(const float* row, int lane) {
  return reinterpret_cast<const float2*>(row)[lane];
}
__device__ __forceinline__ float2 lane_pair(const bf16* row, int lane) {
  const uint32_t v = reinterpret_cast<const uint32_t*>(row)[lane];
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// A lane's pair of a row that starts anywhere, 0 for channels past the last.
template <typename T>
__device__ __forceinline__ float2 any_pair(const T* row, int lane, int cols) {
  return make_float2(2 * lane < cols ? to_f32(row[2 * lane]) : 0.0f, 2 * lane + 1 < cols ? to_f32(row[2 * lane + 1]) : 0.0f);
}

// Row j from p, a step of `step` elements (32 bits: one multiply-add forms the address).
template <typename T>
__device__ __forceinline__ T* row_at(T* p, int step, int j) {
  return p + (long long)step * j;
}

__device__ __forceinline__ void store_if(uint16_t* at, int j, int rows, uint16_t v) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.lt.s32 p, %0, %1;\n\t@p st.global.b16 [%2], %3;\n\t}" ::"r"(j), "r"(rows), "l"(at),
               "h"(v)
               : "memory");
}
// The larger magnitude of two channels, as the bits of a float (from 0x7f800000 on: not finite).
__device__ __forceinline__ uint32_t abs_max(float2 v) {
  return max(__float_as_uint(v.x) & 0x7fffffffu, __float_as_uint(v.y) & 0x7fffffffu);
}
// The same of a lane's pair of a row.
__device__ __forceinline__ uint32_t lane_abs_max(const float* row, int lane) { return abs_max(lane_pair(row, lane)); }
__device__ __forceinline__ uint32_t lane_abs_max(const bf16* row, int lane) {
  const uint32_t w = reinterpret_cast<const uint32_t*>(row)[lane] & 0x7fff7fffu;
  return max(w, w << 16) & 0xffff0000u;
}

__device__ __forceinline__ void store_if(float* at, int j, int rows, float v) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.lt.s32 p, %0, %1;\n\t@p st.global.f32 [%2], %3;\n\t}" ::"r"(j), "r"(rows), "l"(at),
               "f"(v)
               : "memory");
}

// What an 8-bit checkpoint holds of values far out.  A gate counts for its scale
// up to ±256, and e4m3's conversion holds what lies beyond as ±448 at most: its
// sigmoid is 0 or 1 in fp32 from ±104 on, and a mask of the type's lowest value,
// or an infinity, leaves its scale's other channels the steps of a group that
// reaches 256.  x as in act8::storable.
constexpr uint32_t GATE_MAX_BITS = 0x43800000u;     // of 256
__device__ __forceinline__ float storable(float v, bool gate) { return gate ? v : act8::storable(v); }
__device__ __forceinline__ float2 storable(float2 v, bool gate) {
  return make_float2(storable(v.x, gate), storable(v.y, gate));
}

// |v| as bits, 0 for a NaN: an x that is stored has no infinities, and a gate's count like 256.
__device__ __forceinline__ uint32_t counted(float v) {
  const uint32_t bits = __float_as_uint(v) & 0x7fffffffu;
  return bits <= 0x7f800000u ? bits : 0u;
}

// A lane's two channels at `at`, where j < rows (as a predicate, not a branch).
// VEC: both or none exist, on a boundary of two; else `cols` − 2·lane of them.
template <bool VEC>
__device__ __forceinline__ void store_lane(float* at, int j, int rows, int lane, int cols, float2 v) {
  if constexpr (VEC) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.lt.s32 p, %0, %1;\n\t@p st.global.v2.f32 [%2], {%3, %4};\n\t}" ::"r"(j),
                 "r"(2 * lane < cols ? rows : 0), "l"(at), "f"(v.x), "f"(v.y)
                 : "memory");
  } else {
    store_if(at, j, 2 * lane < cols ? rows : 0, v.x);
    store_if(at + 1, j, 2 * lane + 1 < cols ? rows : 0, v.y);
  }
}
template <bool VEC>
__device__ __forceinline__ void store_lane(bf16* at, int j, int rows, int lane, int cols, float2 v) {
  const __nv_bfloat162 w = __float22bfloat162_rn(v);
  if constexpr (VEC) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.lt.s32 p, %0, %1;\n\t@p st.global.b32 [%2], %3;\n\t}" ::"r"(j),
                 "r"(2 * lane < cols ? rows : 0), "l"(at), "r"(*reinterpret_cast<const uint32_t*>(&w))
                 : "memory");
  } else {
    store_if(reinterpret_cast<uint16_t*>(at), j, 2 * lane < cols ? rows : 0, __bfloat16_as_ushort(w.x));
    store_if(reinterpret_cast<uint16_t*>(at) + 1, j, 2 * lane + 1 < cols ? rows : 0, __bfloat16_as_ushort(w.y));
  }
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

// −R2L_GATED_RATE · softplus(lam), log a at an open gate; 0 for channels past the last.
__device__ __forceinline__ float2 decay_rates(const float* lam, int lane, int cols) {
  return make_float2(2 * lane < cols ? decay_rate(lam[2 * lane]) : 0.0f,
                     2 * lane + 1 < cols ? decay_rate(lam[2 * lane + 1]) : 0.0f);
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
// [blocks][LANES] maps and alternates between two buffers from round to round:
// a block writes a buffer again only after the barrier of the round between,
// which every reader of the buffer has passed.
template <int LANES>
__device__ __forceinline__ float2 through_cluster(float4* box, float4 mine, int group, int groups, int lane, uint32_t rank,
                                                  uint32_t blocks, float2& carry) {
  for (uint32_t to = group; to < blocks; to += groups) store_to_rank(box + rank * LANES + lane, to, mine);
  __syncwarp();
  cluster_sync();
  float2 enters = carry;
  for (uint32_t q = 0; q < blocks; ++q) {
    if (q == rank) enters = carry;
    carry = apply(box[q * LANES + lane], carry);
  }
  return enters;
}

// A warp's arrival at the named barrier at which `warp` waits (it alone):
// what it wrote before, the other reads after.  Barrier 0 is __syncthreads'.
__device__ __forceinline__ void pass_to(int warp) { asm volatile("barrier.cta.arrive %0, 64;" ::"r"(1 + warp) : "memory"); }
__device__ __forceinline__ void wait_at(int warp) { asm volatile("barrier.cta.sync %0, 64;" ::"r"(1 + warp) : "memory"); }

// The other half warp's value.
__device__ __forceinline__ float2 other_half(float2 v) {
  return make_float2(__shfl_xor_sync(0xffffffffu, v.x, 16), __shfl_xor_sync(0xffffffffu, v.y, 16));
}

// ---------------------------------------------------------------- forward

constexpr int ROWS = 8;      // consecutive rows of a thread

// Whether rows that start anywhere come in whole pieces.  The 8-bit forward in
// fp32 has no registers to spare: in blocks of 8 warps it spills with them and
// takes 25.8 us of 5 ragged x 777 x 515 (by elements 23.9), 65.6 of 16 x 1000 x
// 515 (58.1) and 122 of 8 x 2000 x 1037 (111).  In blocks of 4 warps pieces are
// ahead all the same (61 x 512 x 1037: 180 us and 186), and so they are in bf16
// (8 x 2000 x 1037: 101 us and 118).
template <typename T, bool VEC, int MODE, int WARPS>
constexpr bool WHOLE_PIECES = !VEC && !(MODE == 2 && sizeof(T) == 4 && WARPS == 8);

// In shared memory, behind it the maps of the cluster's blocks, [2][blocks][LANES].
template <typename T, bool ANY, int LANES, int WARPS>
struct FwdSmem {
  T in[2][3][WARPS * Layout<T, LANES, ROWS, ANY>::WARP_STRIDE];
  float4 maps[2][WARPS][LANES];
  float2 carry[WARPS][LANES];
};
template <typename T, bool ANY, int LANES, int WARPS>
constexpr size_t fwd_smem_bytes(uint32_t blocks) {
  return sizeof(FwdSmem<T, ANY, LANES, WARPS>) + (blocks > 1 ? 2 * sizeof(float4) * LANES * blocks : 0);
}

// MODE 0: the recurrence; 1: also the states of a checkpoint; 2: and its 8 bits.
template <typename T, bool VEC, int MODE, int LANES, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS)
    gated_scan_kernel(const FwdArgs p, const uint32_t blocks) {
  constexpr bool ANY = WHOLE_PIECES<T, VEC, MODE, WARPS>;
  typedef Layout<T, LANES, ROWS, ANY> Lay;
  typedef FwdSmem<T, ANY, LANES, WARPS> Smem;
  static_assert(MODE < 2 || LANES == 32, "the channels of a scale are a row of the warp");
  constexpr int SPAN = WARPS * Lay::WARP_ROWS;      // rows of the block's tile
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  float4* const box = reinterpret_cast<float4*>(smem_raw + sizeof(Smem));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), wl = threadIdx.x & 31;   // uniform for the compiler too
  const int lane = wl % LANES, half = wl / LANES;
  if (p.status && blockIdx.x == 0) write_status(p.lengths, p.B, p.L, p.status);
  const uint32_t rank = blockIdx.x % blocks;
  const uint32_t job = blockIdx.x / blocks;
  const uint32_t strips = (uint32_t)(p.E - 1) / Lay::CHANNELS + 1;
  const int b = (int)(job / strips), e0 = (int)(job % strips) * Lay::CHANNELS, cols = min(p.E - e0, Lay::CHANNELS);
  const int n = clamped_length(p.lengths, b, p.L);
  const int dir = p.forward ? 1 : -1;
  const int span = SPAN * (int)blocks;                 // positions of a round
  const int rounds = n > 0 ? (n - 1) / span + 1 : 0;
  const int k0 = (int)rank * SPAN + warp * Lay::WARP_ROWS;     // this warp's first position in the first round
  const long long row0 = (long long)b * p.L + (p.forward ? 0 : n - 1);   // position 0

  const bool exists = Lay::channel(wl) < cols;       // VEC: this lane's chunk of a row
  const int c0 = e0 + (VEC && exists ? Lay::channel(wl) : 0);
  const T* const x0 = (const T*)p.x + row0 * p.ldx + c0;
  const T* const r0 = (const T*)p.r + row0 * p.ldr + c0;
  const T* const g0 = (const T*)p.g + row0 * p.ldg + c0;
  T* const y0 = (T*)p.y + row0 * p.ldy + e0;
  const int x_step = dir * (int)p.ldx, r_step = dir * (int)p.ldr, g_step = dir * (int)p.ldg, y_step = dir * (int)p.ldy;
  constexpr int ARRAY = WARPS * Lay::WARP_STRIDE;
  T* const rows0 = sm.in[0][0] + warp * Lay::WARP_STRIDE;

  const uint32_t chunk0 = smem_addr(rows0 + Lay::chunk(wl));
  const Edges edges = array_edges(b, p.B, n, p.L, p.forward);
  auto load = [&](int buf, int k) {
    if (k < n) {
      if constexpr (VEC) {
        const uint32_t to = chunk0 + buf * (3 * ARRAY * (int)sizeof(T));
        copy_rows<T, Lay>(to, x0, x_step, k, n, wl, exists);
        copy_rows<T, Lay>(to + ARRAY * (int)sizeof(T), r0, r_step, k, n, wl, exists);
        copy_rows<T, Lay>(to + 2 * ARRAY * (int)sizeof(T), g0, g_step, k, n, wl, exists);
      } else {
        auto copy = [&](T* to, const T* first, int step) {
          if constexpr (ANY) copy_any<T, Lay>(to, first, step, k, n, cols, edges, wl);
          else copy_elements<T, Lay>(to, first, step, k, n, cols, wl);
        };
        T* const to = rows0 + buf * 3 * ARRAY;
        copy(to, x0, x_step);
        copy(to + ARRAY, r0, r_step);
        copy(to + 2 * ARRAY, g0, g_step);
      }
    }
    copies_commit();
  };
  // the first rows are on their way before anything is waited for
  load(0, k0);
  load(1, k0 + span);

  const float2 rate2 = __fmul2_rn(decay_rates(p.lam + e0, lane, cols), two(LOG2E));
  const float2 scale = near_scale(rate2);
  const bool near = __all_sync(0xffffffffu, rate2.x >= NEAR_RATE2 && rate2.y >= NEAR_RATE2);
  float2 carry = p.h0 ? load_vec_pair(p.h0 + (size_t)b * p.E + e0, lane, cols) : two(0.0f);
  if (blocks > 1) cluster_sync();   // every block of the cluster runs before its shared memory is written

  auto scan = [&](auto near_tag) {
    constexpr bool NEAR = decltype(near_tag)::value;
    int k = k0;              // this warp's first position
    for (int round = 0; round < rounds; ++round, k += span) {
      const int buf = round & 1, left = n - k;      // positions from this warp's first one to the end
      const T* const in = rows0 + buf * 3 * ARRAY + half * Lay::GROUP_STRIDE;
      copies_wait<1>();
      __syncwarp();
      // rows that start anywhere: where this group's first ones do (rows past the end are filled from any start)
      const int first = k + half * ROWS, x_offset = !ANY ? 0 : offset_of(x0, x_step, first),
                r_offset = !ANY ? 0 : offset_of(r0, r_step, first), g_offset = !ANY ? 0 : offset_of(g0, g_step, first);
      auto value = [&](int i, int j) {      // x, r or g of row j of this group
        const T* const at = in + i * ARRAY + j * Lay::ROW;
        if constexpr (!ANY) return lane_pair(at, lane);
        const uint32_t offset = (i == 0 ? x_offset : i == 1 ? r_offset : g_offset) +
                                (uint32_t)j * (uint32_t)(i == 0 ? x_step : i == 1 ? r_step : g_step);
        return any_pair(at + (offset & (Lay::PER - 1)), lane, cols);
      };
      float2 P[ROWS], H[ROWS];     // row j's state is P[j] · (state that enters the group) + H[j]
      float2 a = two(1.0f), h = two(0.0f);
      if (left > 0) {
        if (left < Lay::WARP_ROWS) {
          // A position past the end has r = −∞ and x = 0: a = 1, b = 0, and no
          // other test is needed in the arithmetic.
          T* const to = rows0 + buf * 3 * ARRAY;
          fill_rows<T, Lay>(to, wl, left, 0.0f);
          fill_rows<T, Lay>(to + ARRAY, wl, left, -INFINITY);
          fill_rows<T, Lay>(to + 2 * ARRAY, wl, left, 0.0f);
          __syncwarp();
        }
        if constexpr (MODE == 2) {
          // 8-bit copies: the channels that share a scale are one row of the
          // warp.  Lane 8i + j gets the largest magnitude of row j of array i and
          // works out that row's scale; the row's lanes have it by a shuffle.
          const size_t strip = (size_t)b * strips + e0 / Lay::CHANNELS;
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < 3; ++i)
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
              const uint32_t m = __reduce_max_sync(
                    0xffffffffu, !ANY ? lane_abs_max(in + i * ARRAY + j * Lay::ROW, lane) : abs_max(value(i, j)));
              if (lane == i * ROWS + j) top = m;
            }
          const uint32_t most = lane < ROWS ? 0xffffffffu : GATE_MAX_BITS;
          if (top <= 0x7f800000u) top = min(top, most);
          const bool odd = __any_sync(0xffffffffu, top >= act8::SPECIAL);     // a NaN, or an x far out
          if (odd) {
#pragma unroll 1
            for (int c = 0; c < 3 * ROWS; ++c) {
              const float2 v = storable(value(c / ROWS, c % ROWS), c >= ROWS);
              const uint32_t m = __reduce_max_sync(0xffffffffu, max(counted(v.x), counted(v.y)));
              if (lane == c) top = min(m, most);
            }
          }
          const uint32_t byte = act8::scale_byte(top);
          const float down = act8::scale_down(byte);
          if (lane < 3 * ROWS && lane % ROWS < left)
            p.ck.scales[0][lane / ROWS * (p.ck.scales[1] - p.ck.scales[0]) + strip * p.ck.Lp + k + lane % ROWS] = (uint8_t)byte;
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            uint16_t* const q = reinterpret_cast<uint16_t*>(p.ck.q[i] + (strip * p.L + k) * STRIP) + lane;
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
              float2 v = value(i, j);
              if (odd) v = storable(v, i > 0);
              v = __fmul2_rn(v, two(__shfl_sync(0xffffffffu, down, i * ROWS + j)));
              store_if(q + j * (STRIP / 2), j, left, act8::to_e4m3x2(v.x, v.y));
            }
          }
        }
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
          float2 aj, bj;
          coefficients<NEAR>(value(0, j), value(1, j), value(2, j), rate2, scale, aj, bj);
          a = j == 0 ? aj : __fmul2_rn(a, aj);
          h = j == 0 ? bj : __ffma2_rn(aj, h, bj);
          P[j] = a;
          H[j] = h;
        }
      }
      // the warp's map, and what its first half's does to the second half
      float4 map = make_float4(a.x, a.y, h.x, h.y), before = make_float4(1.0f, 1.0f, 0.0f, 0.0f);
      if (Lay::GROUPS == 2) {
        const float2 oa = other_half(a), oh = other_half(h);
        const float4 o = make_float4(oa.x, oa.y, oh.x, oh.y);
        if (half) before = o;
        map = after(half ? map : o, half ? o : map);
      }
      if (blocks > 1 && half == 0) sm.maps[buf][warp][lane] = map;
      __syncwarp();            // the warp has read its rows: their buffer takes the tile after the next
      load(buf, k + 2 * span);
      float2 enters;           // the value that enters this warp
      if (blocks == 1) {
        // from warp to warp, and from the last one to the first one's next rows
        if (round == 0 && warp == 0) {
          enters = carry;
        } else {
          wait_at(warp);
          enters = sm.carry[warp][lane];
        }
        carry = apply(map, enters);
        if (round + 1 < rounds || warp + 1 < WARPS) {
          const int next = (warp + 1) % WARPS;
          if (half == 0) sm.carry[next][lane] = carry;
          __syncwarp();
          pass_to(next);
        }
      } else {
        __syncthreads();
        float4 tile = sm.maps[buf][0][lane];
#pragma unroll
        for (int w = 1; w < WARPS; ++w) tile = after(sm.maps[buf][w][lane], tile);
        enters = through_cluster<LANES>(box + buf * blocks * LANES, tile, warp * Lay::GROUPS + half, WARPS * Lay::GROUPS, lane,
                                        rank, blocks, carry);
        for (int w = 0; w < warp; ++w) enters = apply(sm.maps[buf][w][lane], enters);
      }
      if (MODE >= 1 && k % TILE == 0 && half == 0 && left > 0)
        reinterpret_cast<float2*>(p.ck.states + ((size_t)b * p.ck.tiles + k / TILE) * p.strips * STRIP + e0)[lane] = enters;
      if (Lay::GROUPS == 2) enters = apply(before, enters);
      T* const out = y0 + (long long)(k + half * ROWS) * y_step + 2 * lane;
#pragma unroll
      for (int j = 0; j < ROWS; ++j)
        store_lane<VEC>(row_at(out, y_step, j), j, left - half * ROWS, lane, cols, __ffma2_rn(P[j], enters, H[j]));
    }
  };
  if (near) scan(std::true_type());
  else scan(std::false_type());
  if (p.h_last && rank == 0 && warp == WARPS - 1 && half == 0)
    store_pair<false>(p.h_last + (size_t)b * p.E + e0, lane, cols, carry);
}

// A few positions (a step of decoding): a thread walks its two channels of a
// sequence.  What bounds it is the chain of its loads: a step of 8 x 4096
// channels takes 2.4 us.
template <typename T, bool VEC>
__global__ void __launch_bounds__(128) gated_walk_kernel(const FwdArgs p, const uint32_t blocks /* of a sequence */) {
  if (p.status && blockIdx.x == 0) write_status(p.lengths, p.B, p.L, p.status);
  const int b = (int)(blockIdx.x / blocks), pair = (int)(blockIdx.x % blocks * blockDim.x + threadIdx.x);
  if (2 * pair >= p.E) return;
  const int n = clamped_length(p.lengths, b, p.L);
  const float2 rate2 = __fmul2_rn(decay_rates(p.lam, pair, p.E), two(LOG2E));
  float2 h = p.h0 ? load_vec_pair(p.h0 + (size_t)b * p.E, pair, p.E) : two(0.0f);
  for (int k = 0; k < n; ++k) {
    const long long m = (long long)b * p.L + (p.forward ? k : n - 1 - k);
    float2 aj, bj;
    coefficients<false>(load_pair<VEC>((const T*)p.x + m * p.ldx, pair, p.E), load_pair<VEC>((const T*)p.r + m * p.ldr, pair, p.E),
                        load_pair<VEC>((const T*)p.g + m * p.ldg, pair, p.E), rate2, two(0.0f), aj, bj);
    h = __ffma2_rn(aj, h, bj);
    store_pair<VEC>((T*)p.y + m * p.ldy, pair, p.E, h);
  }
  if (p.h_last) store_pair<false>(p.h_last + (size_t)b * p.E, pair, p.E, h);
}

}  // namespace gated
}  // namespace r2l
