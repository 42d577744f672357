// Kernels of the gated recurrence's gradient (notation of gated_scan.cuh).
//
// A block owns 32 channels of a sequence and takes its tiles from the last to
// the first.  The adjoint of a warp's rows is an affine map of D like their
// states are of h, with the same product of decays, so one exchange between
// the warps hands both on: D from the warps (and the cluster's blocks) behind,
// h from the state saved at the tile's start and the warps before.
#pragma once

#include "gated_scan.cuh"

namespace r2l {
namespace gated {

constexpr float TINY = 1.17549435e-38f;
constexpr int BL = 16;                     // lanes of a row

template <typename T, bool ACT8, int WARPS>
struct BwdSmem {
  typedef typename std::conditional<ACT8, uint8_t, T>::type Q;
  Q in[2][3][WARPS * Layout<Q, BL, ROWS>::WARP_STRIDE];
  T dy[2][WARPS * Layout<T, BL, ROWS>::WARP_STRIDE];
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

template <typename T, bool VEC, bool ACT8, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, (sizeof(T) == 2 ? 16 : 12) / WARPS)
    gated_bwd_kernel(const BwdArgs p, const uint32_t blocks) {
  typedef BwdSmem<T, ACT8, WARPS> Smem;
  typedef typename Smem::Q Q;
  typedef Layout<Q, BL, ROWS> LayQ;
  typedef Layout<T, BL, ROWS> Lay;
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
  // position of this warp's first row in the first round: the last round of the forward, its blocks in reverse
  const long long k0 = (long long)(rounds - 1) * span + (long long)(blocks - 1 - rank) * SPAN + warp * Lay::WARP_ROWS;
  const long long row = (long long)b * p.L + (p.forward ? 0 : n - 1) + dir * k0;
  const float2 rate = decay_rates(p.lam + e0, lane, cols), rate2 = __fmul2_rn(rate, two(LOG2E));
  const float2 k = near_scale(rate2);
  const float2 nik = make_float2(k.x > 0.0f ? -1.0f / k.x : 0.0f, k.y > 0.0f ? -1.0f / k.y : 0.0f);
  const bool near = __all_sync(0xffffffffu, rate2.x >= NEAR_RATE2 && rate2.y >= NEAR_RATE2);
  float2 carry = p.dh_last ? load_vec_pair(p.dh_last + (size_t)b * p.E + e0, lane, cols) : two(0.0f);
  float2 dlam = two(0.0f);

  RowStream<Q, true, LayQ> q0, q1, q2;             // x, r, g of a checkpoint: rows of 64 bytes in scan order
  RowStream<T, VEC, Lay> xs, rs, gs, ds;
  const size_t strip = (size_t)b * p.strips + e0 / STRIP;
  if (ACT8) {
    q0.start(p.ck.q[0], (long long)strip * p.L + k0, STRIP, 1, e0 % STRIP, -span, wl);
    q1.start(p.ck.q[1], (long long)strip * p.L + k0, STRIP, 1, e0 % STRIP, -span, wl);
    q2.start(p.ck.q[2], (long long)strip * p.L + k0, STRIP, 1, e0 % STRIP, -span, wl);
  } else {
    xs.start(p.x, row, p.ldx, dir, e0, -span, wl);
    rs.start(p.r, row, p.ldr, dir, e0, -span, wl);
    gs.start(p.g, row, p.ldg, dir, e0, -span, wl);
  }
  ds.start(p.dy, row, p.ld_dy, dir, e0, -span, wl);
  const long long dx_step = dir * p.ld_dx, dr_step = dir * p.ld_dr, dg_step = dir * p.ld_dg;
  T* dx = (T*)p.dx + row * p.ld_dx + half * ROWS * dx_step + e0 + 2 * lane;
  T* dr = (T*)p.dr + row * p.ld_dr + half * ROWS * dr_step + e0 + 2 * lane;
  T* dg = (T*)p.dg + row * p.ld_dg + half * ROWS * dg_step + e0 + 2 * lane;
  const bool wide = VEC && cols == Lay::CHANNELS;
  constexpr int ARRAY = WARPS * LayQ::WARP_STRIDE, DY = WARPS * Lay::WARP_STRIDE;
  Q* const rows0 = sm.in[0][0] + warp * LayQ::WARP_STRIDE;
  T* const dy0 = sm.dy[0] + warp * Lay::WARP_STRIDE;
  long long kload = k0;      // position of the next rows to load
  auto load = [&](int buf) {
    const int rows = (int)min((long long)Lay::WARP_ROWS, n - kload);
    if (kload >= 0 && rows > 0) {
      Q* const to = rows0 + buf * 3 * ARRAY;
      if (ACT8) {
        if (wl / LayQ::CHUNKS < rows) {
          q0.whole(to, wl);
          q1.whole(to + ARRAY, wl);
          q2.whole(to + 2 * ARRAY, wl);
        }
        if (wl < 3) copy16(sm.scales[buf][warp][wl], p.ck.scales[wl] + strip * p.ck.Lp + kload, 16);
      } else if (wide && rows == Lay::WARP_ROWS) {
        xs.whole((T*)to, wl);
        rs.whole((T*)to + ARRAY, wl);
        gs.whole((T*)to + 2 * ARRAY, wl);
      } else {
        copy_part<T, VEC, Lay>((T*)to, xs.at, xs.step, wl, rows, cols, 0.0f);
        copy_part<T, VEC, Lay>((T*)to + ARRAY, rs.at, rs.step, wl, rows, cols, -INFINITY);
        copy_part<T, VEC, Lay>((T*)to + 2 * ARRAY, gs.at, gs.step, wl, rows, cols, 0.0f);
      }
      if (wide && rows == Lay::WARP_ROWS) ds.whole(dy0 + buf * DY, wl);
      else copy_part<T, VEC, Lay>(dy0 + buf * DY, ds.at, ds.step, wl, rows, cols, 0.0f);
      if (wl < BL / 2)
        copy16(sm.states[buf][warp] + 4 * wl, p.ck.states + ((size_t)b * p.ck.tiles + kload / TILE) * p.strips * STRIP + e0 + 4 * wl, 16);
    }
    kload -= span;
    if (ACT8) {
      q0.at += q0.leap;
      q1.at += q1.leap;
      q2.at += q2.leap;
    } else {
      xs.at += xs.leap;
      rs.at += rs.leap;
      gs.at += gs.leap;
    }
    ds.at += ds.leap;
    copies_commit();
  };

  long long left = n - k0;       // positions from this warp's first one to the end
  load(0);
  load(1);
  if (blocks > 1) cluster_sync();
  for (int round = 0; round < rounds; ++round, left += span) {
    const int buf = round & 1;
    const Q* const in = rows0 + buf * 3 * ARRAY + half * LayQ::GROUP_STRIDE;
    const T* const dy = dy0 + buf * DY + half * Lay::GROUP_STRIDE;
    const int mine = (int)min((long long)ROWS, left - half * ROWS);    // rows of this group (none: ≤ 0)
    copies_wait<1>();
    __syncwarp();
    uint2 scale[3];
    if (ACT8) {
#pragma unroll
      for (int i = 0; i < 3; ++i) scale[i] = *reinterpret_cast<const uint2*>(&sm.scales[buf][warp][i][half * ROWS]);
    }
    auto value = [&](int i, int j) {       // x, r or g of row j of this group
      const Q* const at = in + i * ARRAY + j * LayQ::CHANNELS;
      if constexpr (!ACT8) {
        return lane_pair(at, lane);
      } else {
        const uint32_t word = j < 4 ? scale[i].x : scale[i].y;
        const float2 v = __fmul2_rn(act8::from_e4m3x2(reinterpret_cast<const uint16_t*>(at)[lane]),
                                    two(__uint_as_float((j % 4 ? word >> (8 * (j % 4)) : word) << 24 >> 1)));
        // what is read past the end is neither x = 0 nor a closed gate
        return mine == ROWS ? v : j < mine ? v : two(i == 1 ? -INFINITY : 0.0f);
      }
    };
    // of each row: a, σ(g), and (s, β) for channels near 1, (σ(r), 1 − a²) otherwise
    float2 qa[ROWS], qg[ROWS], qs[ROWS], qb[ROWS];
    float2 a = two(1.0f), h = two(0.0f), D = two(0.0f);
    auto first = [&](auto near_tag) {
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        const float2 x = value(0, j), r = value(1, j), g = value(2, j);
        float2 beta;
        if constexpr (decltype(near_tag)::value) {
          const float2 d = sigmoid_den(r);
          qs[j] = make_float2(rsqrt_approx(d.x), rsqrt_approx(d.y));
          const float2 l2 = __fmul2_rn(__fmul2_rn(qs[j], qs[j]), rate2);
          qa[j] = near_decay(l2);
          qb[j] = beta = __fmul2_rn(__fmul2_rn(qs[j], k), near_beta(l2));
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
    };
    if (left > 0) {
      if (near) first(std::true_type());
      else first(std::false_type());
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
      float2 G[ROWS];
#pragma unroll
      for (int j = ROWS - 1; j >= 0; --j) {
        G[j] = __fadd2_rn(D, lane_pair(dy + j * Lay::CHANNELS, lane));
        D = __fmul2_rn(qa[j], G[j]);
      }
      const bool all = wide && left >= Lay::WARP_ROWS;
      auto second = [&](auto near_tag) {
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
          const float2 x = value(0, j), sgx = __fmul2_rn(qg[j], x);
          float2 sr, beta, nv;      // nv = −σ(r) / β
          if constexpr (decltype(near_tag)::value) {
            sr = __fmul2_rn(qs[j], qs[j]);
            beta = qb[j];
            nv = __fmul2_rn(qs[j], __fmul2_rn(nik, near_beta_inverse(__fmul2_rn(sr, rate2))));
          } else {
            // 0 where the gate is closed (or u subnormal), as is the limit of all that it is part of
            const float2 rb = make_float2(qb[j].x < TINY ? 0.0f : rsqrt_approx(qb[j].x), qb[j].y < TINY ? 0.0f : rsqrt_approx(qb[j].y));
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
          if (all) {
            store_whole_pair(dx + j * dx_step, vdx);
            store_whole_pair(dr + j * dr_step, vdr);
            store_whole_pair(dg + j * dg_step, vdg);
          } else if (j < mine) {
            store_pair<VEC>(dx + j * dx_step - 2 * lane, lane, cols, vdx);
            store_pair<VEC>(dr + j * dr_step - 2 * lane, lane, cols, vdr);
            store_pair<VEC>(dg + j * dg_step - 2 * lane, lane, cols, vdg);
          }
        }
      };
      if (near) second(std::true_type());
      else second(std::false_type());
    }
    dx -= span * dx_step;
    dr -= span * dr_step;
    dg -= span * dg_step;
    __syncwarp();            // the warp has read its rows: their buffer takes the tile after the next
    load(buf);
  }
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

// dlam from the blocks' shares, [rows][width]: 8 threads a channel take every
// eighth row each, and their sums are added in order.
__global__ void __launch_bounds__(256) gated_dlam_kernel(const float* part, int rows, int width, const float* lam, int E,
                                                         float* dlam) {
  __shared__ float sum[8][32];
  const int c = threadIdx.x & 31, w = threadIdx.x >> 5, e = blockIdx.x * 32 + c;
  float s = 0.0f;
#pragma unroll 4
  for (int i = w; i < rows; i += 8) s += part[(size_t)i * width + e];
  sum[w][c] = s;
  __syncthreads();
  if (w == 0 && e < E) {
#pragma unroll
    for (int k = 1; k < 8; ++k) s += sum[k][c];
    dlam[e] = s * (-R2L_GATED_RATE / (1.0f + expf(-lam[e])));
  }
}

}  // namespace gated
}  // namespace r2l
