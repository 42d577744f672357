// Kernels of the gated recurrence's gradient (notation of gated_scan.cuh).
//
// A block owns 32 channels of a sequence and takes its tiles from the last to
// the first.  The adjoint of a warp's rows is an affine map of D like their
// states are of h, with the same product of decays, so one exchange between
// the warps hands both on: D from the warps (and the cluster's blocks) behind,
// h from the state saved at the tile's start and the warps before.  A thread
// keeps its 8 rows' gates in registers between the two.
//
// What bounds it (B200, bf16, 8 x 4096 x 4096): 14 bytes per position and
// channel, 288 us at the measured copy rate, against 72 instructions per 32 of
// them at 16 warps an SM (the 128 registers of the gates), of which 65% of the
// issue slots are used: 397 us, 4.8 TB/s.  In fp32 (8 x 2048 x 4096) 313 us,
// 6.0 TB/s.  From 8-bit rows it reads 3 bytes less and spends 14 instructions
// more on them: 445 us.  168 registers and 12 warps: 422 us.  Gradients staged
// in shared memory and written 16 bytes a lane: 407 us.  Rows that start anywhere
// are copied element by element; whole pieces were measured in fp32 alone, in
// blocks bound to 128 registers (5 ragged x 777 x 515: 27 us, and 44 with pieces).
#pragma once

#include "gated_scan.cuh"

namespace r2l {
namespace gated {

constexpr float TINY = 1.17549435e-38f;
constexpr int BL = 16;                     // lanes of a row

template <typename T, bool ACT8, int WARPS>
struct BwdSmem {
  typedef typename std::conditional<ACT8, uint8_t, T>::type Q;
  Q in[2][3][WARPS * Layout<Q, BL, ROWS, false>::WARP_STRIDE];
  T dy[2][WARPS * Layout<T, BL, ROWS, false>::WARP_STRIDE];
  uint8_t scales[2][WARPS][3][2 * ROWS];
  float states[2][WARPS][2 * BL];          // each warp's copy of its 64 positions' first state
  float4 maps[2][WARPS][BL];               // D leaves = A · D enters + B
  float2 h[2][WARPS][BL];                  // h leaves = A · h enters + this
  float2 carry[2][BL];
};
template <typename T, bool ACT8, int WARPS>
constexpr size_t bwd_smem_bytes(uint32_t blocks) {
  return sizeof(BwdSmem<T, ACT8, WARPS>) + (blocks > 1 ? 2 * sizeof(float4) * BL * blocks : 0);
}

// 1 / √((1 − 2^(2 l2)) / (−2 ln 2 · l2)) for −0.5 ≤ l2 ≤ 0 (relative error under 2^-24)
__device__ __forceinline__ float2 near_beta_inverse(float2 l2) {
  float2 c = __ffma2_rn(l2, two(0.00710895564f), two(0.0200518221f));
  c = __ffma2_rn(c, l2, two(-0.346571386f));
  return __ffma2_rn(c, l2, two(1.0f));
}

// Warps of an SM that a thread's registers have to leave room for.  fp32 rows of
// 8 warps fill 145 KB of shared memory, so one block is all that an SM holds,
// whatever its registers: where rows start anywhere it may have them all (246,
// and no spills; 16 x 1000 x 515: 88 -> 78 us, 5 ragged x 777 x 515: 26.8 -> 25.8);
// on 16-byte boundaries 128 are enough (8 x 2048 x 4096: 310 us, and 312 with 252).
template <typename T, bool VEC, bool ACT8, int WARPS>
constexpr int BWD_WARPS = sizeof(T) == 2 ? 16 : WARPS == 4 ? 12 : ACT8 || VEC ? 16 : 8;

template <typename T, bool VEC, bool ACT8, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, BWD_WARPS<T, VEC, ACT8, WARPS> / WARPS)
    gated_bwd_kernel(const BwdArgs p, const uint32_t blocks) {
  typedef BwdSmem<T, ACT8, WARPS> Smem;
  typedef typename Smem::Q Q;
  typedef Layout<Q, BL, ROWS, false> LayQ;
  typedef Layout<T, BL, ROWS, false> Lay;
  constexpr int SPAN = WARPS * Lay::WARP_ROWS, TILE_WARPS = TILE / Lay::WARP_ROWS;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  float4* const box = reinterpret_cast<float4*>(smem_raw + sizeof(Smem));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), wl = threadIdx.x & 31;
  const int lane = wl % BL, half = wl / BL;
  if (blockIdx.x == 0) write_status(p.lengths, p.B, p.L, p.status);
  const uint32_t rank = blockIdx.x % blocks;
  const uint32_t job = blockIdx.x / blocks;
  const uint32_t strips = (uint32_t)(p.E - 1) / Lay::CHANNELS + 1;
  const int b = (int)(job / strips), e0 = (int)(job % strips) * Lay::CHANNELS, cols = min(p.E - e0, Lay::CHANNELS);
  const int n = clamped_length(p.lengths, b, p.L);
  const int dir = p.forward ? 1 : -1;
  const int span = SPAN * (int)blocks;
  const int rounds = n > 0 ? (n - 1) / span + 1 : 0;
  // this warp's first position in the first round: the last round of the forward, its blocks in reverse
  const int k0 = (rounds - 1) * span + (int)(blocks - 1 - rank) * SPAN + warp * Lay::WARP_ROWS;
  const long long row0 = (long long)b * p.L + (p.forward ? 0 : n - 1);   // position 0
  const size_t strip = (size_t)b * p.strips + e0 / STRIP;
  const bool exists = Lay::channel(wl) < cols;       // VEC: this lane's chunk of a row
  const int c0 = exists ? Lay::channel(wl) : 0;
  const Q* in0[3];          // x, r, g: position 0
  int in_step[3];
  if constexpr (ACT8) {     // rows of 64 bytes in scan order
#pragma unroll
    for (int i = 0; i < 3; ++i) in0[i] = p.ck.q[i] + strip * p.L * STRIP + e0 % STRIP, in_step[i] = STRIP;
  } else {
    in0[0] = (const T*)p.x + row0 * p.ldx + e0, in_step[0] = dir * (int)p.ldx;
    in0[1] = (const T*)p.r + row0 * p.ldr + e0, in_step[1] = dir * (int)p.ldr;
    in0[2] = (const T*)p.g + row0 * p.ldg + e0, in_step[2] = dir * (int)p.ldg;
  }
  const T* const first_dy = (const T*)p.dy + row0 * p.ld_dy + e0;
  T* const dx0 = (T*)p.dx + row0 * p.ld_dx + e0;
  T* const dr0 = (T*)p.dr + row0 * p.ld_dr + e0;
  T* const dg0 = (T*)p.dg + row0 * p.ld_dg + e0;
  const float* const states0 = p.ck.states + (long long)b * p.ck.tiles * p.strips * STRIP + e0;
  const int dy_step = dir * (int)p.ld_dy, dx_step = dir * (int)p.ld_dx, dr_step = dir * (int)p.ld_dr, dg_step = dir * (int)p.ld_dg;
  constexpr int ARRAY = WARPS * LayQ::WARP_STRIDE, DY = WARPS * Lay::WARP_STRIDE;
  Q* const rows0 = sm.in[0][0] + warp * LayQ::WARP_STRIDE;
  T* const dy0 = sm.dy[0] + warp * Lay::WARP_STRIDE;

  auto load = [&](int buf, int k) {
    if (k >= 0 && k < n) {
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        Q* const to = rows0 + (buf * 3 + i) * ARRAY;
        if constexpr (ACT8)
          copy_rows<Q, LayQ>(smem_addr(to + LayQ::chunk(wl)), in0[i] + LayQ::channel(wl), in_step[i], k, n, wl, true);
        else if constexpr (VEC)
          copy_rows<Q, LayQ>(smem_addr(to + LayQ::chunk(wl)), in0[i] + c0, in_step[i], k, n, wl, exists);
        else
          copy_elements<Q, LayQ>(to, in0[i], in_step[i], k, n, cols, wl);
      }
      T* const to = dy0 + buf * DY;
      if constexpr (VEC) copy_rows<T, Lay>(smem_addr(to + Lay::chunk(wl)), first_dy + c0, dy_step, k, n, wl, exists);
      else copy_elements<T, Lay>(to, first_dy, dy_step, k, n, cols, wl);
      if (wl < BL / 2)
        copy16(smem_addr(sm.states[buf][warp] + 4 * wl), states0 + (long long)(k / TILE) * (p.strips * STRIP) + 4 * wl);
      if (ACT8 && wl < 3) copy16(smem_addr(sm.scales[buf][warp][wl]), p.ck.scales[wl] + strip * p.ck.Lp + k);
    }
    copies_commit();
  };
  // the first rows are on their way before anything is waited for
  load(0, k0);
  load(1, k0 - span);

  const float2 rate = decay_rates(p.lam + e0, lane, cols), rate2 = __fmul2_rn(rate, two(LOG2E));
  const float2 scale = near_scale(rate2);
  const float2 nscale = make_float2(scale.x > 0.0f ? -1.0f / scale.x : 0.0f, scale.y > 0.0f ? -1.0f / scale.y : 0.0f);
  const bool near = __all_sync(0xffffffffu, rate2.x >= NEAR_RATE2 && rate2.y >= NEAR_RATE2);
  float2 carry = p.dh_last ? load_vec_pair(p.dh_last + (size_t)b * p.E + e0, lane, cols) : two(0.0f);
  float2 dlam = two(0.0f);
  if (blocks > 1) cluster_sync();

  auto walk = [&](auto near_tag) {
    constexpr bool NEAR = decltype(near_tag)::value;
    int k = k0;                    // this warp's first position
    for (int round = 0; round < rounds; ++round, k -= span) {
      const int buf = round & 1, left = n - k;     // positions from this warp's first one to the end
      const Q* const in = rows0 + buf * 3 * ARRAY + half * LayQ::GROUP_STRIDE;
      const T* const dy = dy0 + buf * DY + half * Lay::GROUP_STRIDE;
      const int mine = min(ROWS, left - half * ROWS);    // rows of this group (none: ≤ 0)
      copies_wait<1>();
      __syncwarp();
      uint2 factors[3];
      if (ACT8) {
#pragma unroll
        for (int i = 0; i < 3; ++i) factors[i] = *reinterpret_cast<const uint2*>(&sm.scales[buf][warp][i][half * ROWS]);
      }
      auto value = [&](int i, int j) {       // x, r or g of row j of this group
        const Q* const at = in + i * ARRAY + j * LayQ::CHANNELS;
        if constexpr (!ACT8) {
          return lane_pair(at, lane);
        } else {
          const uint32_t word = j < 4 ? factors[i].x : factors[i].y;
          const float2 v = __fmul2_rn(act8::from_e4m3x2(reinterpret_cast<const uint16_t*>(at)[lane]),
                                      two(__uint_as_float((j % 4 ? word >> (8 * (j % 4)) : word) << 24 >> 1)));
          // what is read past the end is neither x = 0 nor a closed gate
          return mine == ROWS ? v : j < mine ? v : two(i == 1 ? -INFINITY : 0.0f);
        }
      };
      // of each row: a, σ(g), and (s, β) for channels near 1, (σ(r), 1 − a²) otherwise
      float2 qa[ROWS], qg[ROWS], qs[ROWS], qb[ROWS];
      float2 a = two(1.0f), h = two(0.0f), D = two(0.0f);
      if (left > 0) {
        if (left < Lay::WARP_ROWS) {
          // a position past the end has r = −∞, x = 0 and dy = 0
          if constexpr (!ACT8) {
            T* const to = (T*)rows0 + buf * 3 * ARRAY;
            fill_rows<T, Lay>(to, wl, left, 0.0f);
            fill_rows<T, Lay>(to + ARRAY, wl, left, -INFINITY);
            fill_rows<T, Lay>(to + 2 * ARRAY, wl, left, 0.0f);
          }
          fill_rows<T, Lay>(dy0 + buf * DY, wl, left, 0.0f);
          __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
          const float2 x = value(0, j), r = value(1, j), g = value(2, j);
          float2 beta;
          if constexpr (NEAR) {
            const float2 d = sigmoid_den(r);
            qs[j] = make_float2(rsqrt_approx(d.x), rsqrt_approx(d.y));
            const float2 l2 = __fmul2_rn(__fmul2_rn(qs[j], qs[j]), rate2);
            qa[j] = near_decay(l2);
            qb[j] = beta = __fmul2_rn(__fmul2_rn(qs[j], scale), near_beta(l2));
            qg[j] = sigmoid2(g);
          } else {
            const Gates q = gates2(r, g, rate2);
            qa[j] = q.a;
            qg[j] = q.sg;
            qs[j] = q.sr;
            qb[j] = q.u;
            beta = make_float2(sqrt_approx(q.u.x), sqrt_approx(q.u.y));
          }
          h = __ffma2_rn(qa[j], h, __fmul2_rn(beta, __fmul2_rn(qg[j], x)));
          a = j == 0 ? qa[j] : __fmul2_rn(a, qa[j]);
        }
#pragma unroll
        for (int j = ROWS - 1; j >= 0; --j) D = __fmul2_rn(qa[j], __fadd2_rn(D, lane_pair(dy + j * Lay::CHANNELS, lane)));
      }
      const float2 oa = other_half(a), oh = other_half(h), oD = other_half(D);
      if (half == 0) {
        const float4 map = after(make_float4(a.x, a.y, D.x, D.y), make_float4(oa.x, oa.y, oD.x, oD.y));
        sm.maps[buf][warp][lane] = map;
        sm.h[buf][warp][lane] = __ffma2_rn(oa, h, oh);
      }
      __syncthreads();
      if (blocks > 1) {
        float4 tile = sm.maps[buf][WARPS - 1][lane];
#pragma unroll
        for (int w = WARPS - 2; w >= 0; --w) tile = after(sm.maps[buf][w][lane], tile);
        D = through_cluster<BL>(box + buf * blocks * BL, tile, warp * 2 + half, WARPS * 2, lane, rank, blocks, carry);
      } else {
        D = round == 0 ? carry : sm.carry[buf ^ 1][lane];
      }
      for (int w = WARPS - 1; w > warp; --w) D = apply(sm.maps[buf][w][lane], D);
      if (blocks == 1 && warp == 0) {
        carry = apply(sm.maps[buf][0][lane], D);
        if (half == 0) sm.carry[buf][lane] = carry;
      }
      if (left > 0) {
        h = reinterpret_cast<const float2*>(sm.states[buf][warp])[lane];
        for (int w = warp / TILE_WARPS * TILE_WARPS; w < warp; ++w) {
          const float4 m = sm.maps[buf][w][lane];
          h = __ffma2_rn(make_float2(m.x, m.y), h, sm.h[buf][w][lane]);
        }
        if (half) h = __ffma2_rn(oa, h, oh);
        else D = __ffma2_rn(oa, D, oD);
        T* const dx = dx0 + (long long)(k + half * ROWS) * dx_step + 2 * lane;
        T* const dr = dr0 + (long long)(k + half * ROWS) * dr_step + 2 * lane;
        T* const dg = dg0 + (long long)(k + half * ROWS) * dg_step + 2 * lane;
        float2 G[ROWS];
#pragma unroll
        for (int j = ROWS - 1; j >= 0; --j) {
          G[j] = __fadd2_rn(D, lane_pair(dy + j * Lay::CHANNELS, lane));
          D = __fmul2_rn(qa[j], G[j]);
        }
#pragma unroll
          for (int j = 0; j < ROWS; ++j) {
            const float2 x = value(0, j), sgx = __fmul2_rn(qg[j], x);
            float2 sr, beta, nv;      // nv = −σ(r) / β
            if constexpr (NEAR) {
              sr = __fmul2_rn(qs[j], qs[j]);
              beta = qb[j];
              nv = __fmul2_rn(qs[j], __fmul2_rn(nscale, near_beta_inverse(__fmul2_rn(sr, rate2))));
            } else {
              // 0 where the gate is closed (or u subnormal), as is the limit of all that it is part of
              const float2 rb = make_float2(qb[j].x < TINY ? 0.0f : rsqrt_approx(qb[j].x),
                                            qb[j].y < TINY ? 0.0f : rsqrt_approx(qb[j].y));
              sr = make_float2(qb[j].x < TINY ? 0.0f : qs[j].x, qb[j].y < TINY ? 0.0f : qs[j].y);
              beta = __fmul2_rn(qb[j], rb);
              nv = __fmul2_rn(__fmul2_rn(sr, rb), two(-1.0f));
            }
            const float2 vdx = __fmul2_rn(G[j], __fmul2_rn(beta, qg[j]));
            const float2 vdg = __fmul2_rn(__fmul2_rn(vdx, x), __ffma2_rn(qg[j], two(-1.0f), two(1.0f)));
            // d(log a) σ(r) = G a (h σ(r) − σ(g) x a σ(r) / β)
            const float2 t = __ffma2_rn(sgx, __fmul2_rn(qa[j], nv), __fmul2_rn(h, sr));
            const float2 dls = __fmul2_rn(__fmul2_rn(G[j], qa[j]), t);
            dlam = __fadd2_rn(dlam, dls);
            const float2 vdr = __fmul2_rn(__fmul2_rn(dls, rate), __ffma2_rn(sr, two(-1.0f), two(1.0f)));
            h = __ffma2_rn(qa[j], h, __fmul2_rn(beta, sgx));
            store_lane<VEC>(row_at(dx, dx_step, j), j, mine, lane, cols, vdx);
            store_lane<VEC>(row_at(dr, dr_step, j), j, mine, lane, cols, vdr);
            store_lane<VEC>(row_at(dg, dg_step, j), j, mine, lane, cols, vdg);
        }
      }
      __syncwarp();            // the warp has read its rows: their buffer takes the tile after the next
      load(buf, k - 2 * span);
    }
  };
  if (near) walk(std::true_type());
  else walk(std::false_type());
  if (p.dh0 && rank == 0 && warp == 0 && half == 0) store_pair<false>(p.dh0 + (size_t)b * p.E + e0, lane, cols, carry);
  for (long long i = n + (long long)(rank * WARPS + warp) * 2 + half; i < p.L; i += blocks * WARPS * 2) {   // rows past the end
    const long long m = (long long)b * p.L + i;
    store_pair<VEC>((T*)p.dx + m * p.ld_dx + e0, lane, cols, two(0.0f));
    store_pair<VEC>((T*)p.dr + m * p.ld_dr + e0, lane, cols, two(0.0f));
    store_pair<VEC>((T*)p.dg + m * p.ld_dg + e0, lane, cols, two(0.0f));
  }
  // this block's share of dlam: its groups in order
  __syncthreads();
  const float2 od = other_half(dlam);
  if (half == 0) sm.h[0][warp][lane] = __fadd2_rn(dlam, od);
  __syncthreads();
  if (warp == 0 && half == 0) {
    dlam = sm.h[0][0][lane];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) dlam = __fadd2_rn(dlam, sm.h[0][w][lane]);
    reinterpret_cast<float2*>(p.part + ((size_t)b * blocks + rank) * p.strips * STRIP + e0)[lane] = dlam;
  }
}

// Sums of the blocks' shares of dlam, [rows][width]: a block takes 32 channels
// of `per` rows, 8 threads a channel every eighth of them, and their sums are
// added in order.  Into out[blockIdx.y][width], or where lam is given into
// dlam, times its derivative.
constexpr int DLAM_ROWS = 1024;     // rows of a block; more are summed in two launches
__global__ void __launch_bounds__(256) gated_dlam_kernel(const float* part, int rows, int per, int width, const float* lam,
                                                         int E, float* out) {
  __shared__ float sum[8][32];
  const int c = threadIdx.x & 31, w = threadIdx.x >> 5, e = blockIdx.x * 32 + c;
  const int from = blockIdx.y * per, to = min(rows, from + per);
  float s = 0.0f;
#pragma unroll 4
  for (int i = from + w; i < to; i += 8) s += part[(size_t)i * width + e];
  sum[w][c] = s;
  __syncthreads();
  if (w != 0) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) s += sum[k][c];
  if (!lam) out[(size_t)blockIdx.y * width + e] = s;
  else if (e < E) out[e] = s * (-R2L_GATED_RATE / (1.0f + expf(-lam[e])));
}

}  // namespace gated
}  // namespace r2l
