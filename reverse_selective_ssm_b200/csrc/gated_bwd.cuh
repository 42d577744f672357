// Kernels of the gated recurrence's gradient (notation of gated_scan.cuh).
//
// A block owns 64 channels of a sequence and takes its tiles from the last to
// the first.  A tile's adjoint is an affine map of D like its states are of h,
// with the same product of decays, so one exchange between the warps hands
// both on: D from the warps (and the cluster's blocks) behind, h from the
// state saved at the tile's start and the warps before.
#pragma once

#include <type_traits>

#include "gated_scan.cuh"

namespace r2l {
namespace gated {

constexpr int BW = 8;              // warps of a gradient block
constexpr int BP = TILE / BW;      // rows of a warp
constexpr float TINY = 1.17549435e-38f;

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

template <typename T, bool ACT8>
struct BwdSmem {
  typedef typename std::conditional<ACT8, uint8_t, T>::type Q;
  Q in[2][3][TILE * STRIP];
  T dy[2][TILE * STRIP];
  float states[2][STRIP];
  uint8_t scales[2][3][TILE];
  float4 maps[BW][32];             // D leaves = A · D enters + B
  float2 h[BW][32];                // h leaves = A · h enters + this
};

__device__ __forceinline__ float2 lane_pair8(const uint8_t* row, int lane, uint32_t scale) {
  return __fmul2_rn(act8::from_e4m3x2(reinterpret_cast<const uint16_t*>(row)[lane]), two(act8::scale_up(scale)));
}

constexpr size_t box_bytes(uint32_t blocks) { return blocks > 1 ? 2 * (size_t)blocks * 32 * sizeof(float4) : 0; }

template <typename T, bool VEC, bool ACT8>
__global__ void __launch_bounds__(BW * 32, 2) gated_bwd_kernel(const BwdArgs p, const uint32_t blocks) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  BwdSmem<T, ACT8>& sm = *reinterpret_cast<BwdSmem<T, ACT8>*>(smem_raw);
  float4* const box = reinterpret_cast<float4*>(smem_raw + sizeof(BwdSmem<T, ACT8>));
  if (blockIdx.x == 0) write_status(p.lengths, p.B, p.L, p.status);
  const uint32_t rank = blockIdx.x % blocks;
  const uint32_t job = blockIdx.x / blocks;
  const int strip = (int)(job % (uint32_t)p.strips), b = (int)(job / (uint32_t)p.strips);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int e0 = strip * STRIP, cols = min(p.E - e0, STRIP);
  const int n = clamped_length(p.lengths, b, p.L);
  const long long row0 = (long long)b * p.L + (p.forward ? 0 : n - 1);
  const int dir = p.forward ? 1 : -1;
  const float2 rate = decay_rates(p.lam + e0, lane, cols), rate2 = __fmul2_rn(rate, two(LOG2E));
  float2 carry = p.dh_last ? load_vec_pair(p.dh_last + (size_t)b * p.E + e0, lane, cols) : two(0.0f);
  float2 dlam = two(0.0f);

  const int tiles = (n + TILE - 1) / TILE;
  const int rounds = (tiles + (int)blocks - 1) / (int)blocks;
  // block 0 of the cluster takes the last tile of a round
  auto load = [&](int round) {
    const int tile = tiles - 1 - round * (int)blocks - (int)rank, buf = round & 1;
    if (tile >= 0) {
      const long long k0 = (long long)tile * TILE;
      const int rows = (int)min((long long)TILE, n - k0);
      if (ACT8) {
        const size_t at = ((size_t)b * p.strips + strip) * p.L + k0;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const int row = threadIdx.x / 4, c = threadIdx.x % 4 * 16;   // 256 threads, 64 rows of 64 bytes
          if (row < rows)
            copy16((uint8_t*)sm.in[buf][i] + row * STRIP + c, p.ck.q[i] + (at + row) * STRIP + c, 16);
        }
        if (threadIdx.x < 12) {   // 64 bytes of scales each; the padding of their rows covers a part tile
          const int i = threadIdx.x / 4, c = threadIdx.x % 4 * 16;
          if (c < rows)
            copy16(sm.scales[buf][i] + c, p.ck.scales[i] + ((size_t)b * p.strips + strip) * p.ck.Lp + k0 + c, 16);
        }
      } else {
        load_tile<T, VEC, BW * 32>((T*)sm.in[buf][0], (const T*)p.x + (row0 + dir * k0) * p.ldx + e0, dir * p.ldx, rows, cols, 0.0f);
        load_tile<T, VEC, BW * 32>((T*)sm.in[buf][1], (const T*)p.r + (row0 + dir * k0) * p.ldr + e0, dir * p.ldr, rows, cols, -INFINITY);
        load_tile<T, VEC, BW * 32>((T*)sm.in[buf][2], (const T*)p.g + (row0 + dir * k0) * p.ldg + e0, dir * p.ldg, rows, cols, 0.0f);
      }
      load_tile<T, VEC, BW * 32>(sm.dy[buf], (const T*)p.dy + (row0 + dir * k0) * p.ld_dy + e0, dir * p.ld_dy, rows, cols, 0.0f);
      if (threadIdx.x < 16)
        copy16(sm.states[buf] + threadIdx.x * 4,
               p.ck.states + ((size_t)b * p.ck.tiles + tile) * p.strips * STRIP + e0 + threadIdx.x * 4, 16);
    }
    copies_commit();
  };

  if (rounds > 0) load(0);
  if (rounds > 1) load(1);
  else copies_commit();
  if (blocks > 1) cluster_sync();
  for (int round = 0; round < rounds; ++round) {
    const int buf = round & 1;
    const int tile = tiles - 1 - round * (int)blocks - (int)rank;
    const long long k0 = (long long)tile * TILE;
    const int rows = tile < 0 ? 0 : (int)min((long long)TILE, n - k0);
    const int mine = rows - warp * BP;
    copies_wait<1>();
    __syncthreads();
    auto in = [&](int i, int j) {   // x, r or g of row j of this warp
      const int at = (warp * BP + j) * STRIP;
      if (!ACT8) return lane_pair((const T*)sm.in[buf][i] + at, lane);
      // rows past the end have no closed gate in 8 bits
      return j < mine ? lane_pair8((const uint8_t*)sm.in[buf][i] + at, lane, sm.scales[buf][i][warp * BP + j])
                      : two(i == 1 ? -INFINITY : 0.0f);
    };
    Gates q[BP];
    float2 a = two(1.0f), h = two(0.0f), D = two(0.0f);
    if (mine > 0) {
#pragma unroll
      for (int j = 0; j < BP; ++j) {
        q[j] = gates2(in(1, j), in(2, j), rate2);
        const float2 bx = __fmul2_rn(make_float2(sqrt_approx(q[j].u.x), sqrt_approx(q[j].u.y)), __fmul2_rn(q[j].sg, in(0, j)));
        h = __ffma2_rn(q[j].a, h, bx);
        a = __fmul2_rn(a, q[j].a);
      }
#pragma unroll
      for (int j = BP - 1; j >= 0; --j)
        D = __fmul2_rn(q[j].a, __fadd2_rn(D, lane_pair(sm.dy[buf] + (warp * BP + j) * STRIP, lane)));
    }
    sm.maps[warp][lane] = make_float4(a.x, a.y, D.x, D.y);
    sm.h[warp][lane] = h;
    __syncthreads();
    if (blocks > 1) {
      float4 whole = sm.maps[BW - 1][lane];
#pragma unroll
      for (int w = BW - 2; w >= 0; --w) whole = after(sm.maps[w][lane], whole);
      D = through_cluster(box + buf * blocks * 32, whole, warp, BW, lane, 32, rank, blocks, carry);
    } else {
      D = carry;
#pragma unroll
      for (int w = BW - 1; w >= 0; --w) carry = apply(sm.maps[w][lane], carry);
    }
    if (mine > 0) {
#pragma unroll
      for (int w = BW - 1; w > 0; --w)
        if (w > warp) D = apply(sm.maps[w][lane], D);
      h = reinterpret_cast<const float2*>(sm.states[buf])[lane];
#pragma unroll
      for (int w = 0; w < BW - 1; ++w)
        if (w < warp) {
          const float4 m = sm.maps[w][lane];
          h = __ffma2_rn(make_float2(m.x, m.y), h, sm.h[w][lane]);
        }
      float2 G[BP];
#pragma unroll
      for (int j = BP - 1; j >= 0; --j) {
        G[j] = __fadd2_rn(D, lane_pair(sm.dy[buf] + (warp * BP + j) * STRIP, lane));
        D = __fmul2_rn(q[j].a, G[j]);
      }
      const long long m0 = row0 + dir * (k0 + warp * BP);
      T* const dx = (T*)p.dx + m0 * p.ld_dx + e0;
      T* const dr = (T*)p.dr + m0 * p.ld_dr + e0;
      T* const dg = (T*)p.dg + m0 * p.ld_dg + e0;
#pragma unroll
      for (int j = 0; j < BP; ++j) {
        const float2 x = in(0, j), sr = q[j].sr, sg = q[j].sg, u = q[j].u;
        // 1/β, and 0 where the gate is closed (or u subnormal): all that 1/β multiplies is 0 in the limit
        const float2 rs = make_float2(u.x < TINY ? 0.0f : rsqrt_approx(u.x), u.y < TINY ? 0.0f : rsqrt_approx(u.y));
        const float2 beta = __fmul2_rn(u, rs), sgx = __fmul2_rn(sg, x);
        const float2 vdx = __fmul2_rn(G[j], __fmul2_rn(beta, sg));
        const float2 vdg = __fmul2_rn(__fmul2_rn(vdx, x), __ffma2_rn(sg, two(-1.0f), two(1.0f)));
        // d(log a) = G a (h − σ(g) x a / β)
        const float2 ah = __ffma2_rn(__fmul2_rn(sgx, rs), make_float2(-q[j].a.x, -q[j].a.y), h);
        float2 dl = __fmul2_rn(__fmul2_rn(G[j], q[j].a), ah);
        dl = make_float2(u.x < TINY ? 0.0f : dl.x, u.y < TINY ? 0.0f : dl.y);
        const float2 ds = __fmul2_rn(dl, sr);
        dlam = __fadd2_rn(dlam, ds);
        const float2 vdr = __fmul2_rn(__fmul2_rn(ds, rate), __ffma2_rn(sr, two(-1.0f), two(1.0f)));
        h = __ffma2_rn(q[j].a, h, __fmul2_rn(beta, sgx));
        if (j < mine) {
          store_pair<VEC>(dx + j * dir * p.ld_dx, lane, cols, vdx);
          store_pair<VEC>(dr + j * dir * p.ld_dr, lane, cols, vdr);
          store_pair<VEC>(dg + j * dir * p.ld_dg, lane, cols, vdg);
        }
      }
    }
    __syncthreads();   // this round's rows are read: their buffer may be filled again
    if (round + 2 < rounds) load(round + 2);
    else copies_commit();
  }
  if (p.dh0 && rank == 0 && warp == 0) store_pair<false>(p.dh0 + (size_t)b * p.E + e0, lane, cols, carry);
  for (long long i = n + (long long)rank * BW + warp; i < p.L; i += blocks * BW) {   // rows past the end
    const long long m = (long long)b * p.L + i;
    store_pair<VEC>((T*)p.dx + m * p.ld_dx + e0, lane, cols, two(0.0f));
    store_pair<VEC>((T*)p.dr + m * p.ld_dr + e0, lane, cols, two(0.0f));
    store_pair<VEC>((T*)p.dg + m * p.ld_dg + e0, lane, cols, two(0.0f));
  }
  // this block's share of dlam: its warps in order
  sm.h[warp][lane] = dlam;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int w = 1; w < BW; ++w) dlam = __fadd2_rn(dlam, sm.h[w][lane]);
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
