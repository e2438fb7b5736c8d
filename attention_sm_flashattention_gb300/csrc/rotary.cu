// Rotary positions: pair j of a head's first `rot` values is turned by the
// angle position * freq_j,
//   y0 = m (x0 cos a - x1 sin a),   y1 = m (x1 cos a + x0 sin a),
// the pairs being (j, j + rot / 2) or, interleaved, (2 j, 2 j + 1); values
// past `rot` are copied.  The gradients' way back is the same with -a.  The
// serving form writes the turned keys, and the values, into a paged cache.
//
// The angle in turns is kept as a 64-bit fixed-point fraction: freq / 2 pi is
// rounded to 53 bits once, and its product with the position modulo 2^64 is
// the fraction of a turn, exact for any position (the rounding grows by
// position * 2^-54 of a turn).  Its top 32 bits, as half turns in [-1, 1), go
// through sincospif in fp32: no reduction of a large argument, no table to
// read and no bound on the position.
//
// HBM-bound: every value is read and written once.  A thread owns 8 pairs (two
// 16-byte chunks) of one token, takes their sines and cosines into registers
// and walks over the heads with them, so the angles cost one sincospif per
// pair and token whatever the number of heads.  16 tokens per block at D =
// 128 write 4 KB runs in the [Z, heads, N, D] layout from [Z, N, heads, D]
// rows.  Few tokens: the heads are dealt over the grid's y.
//
// The fractions are formed once per block, one thread per pair: double
// precision runs at about a sixtieth of fp32's rate here, and forming them in
// every thread was most of a small call's time (kernel time 15.7 -> 9.7 us for
// 25 MB at Z3 H16/16 N1021 D64 rot 16; 23 -> 17.3 us for the cache form at
// Z8 H32/8 N512 D128 rot 64).  Z4 H32/8 N8192 D128: 105 us, 6.4 TB/s.
#include <cmath>
#include <cstdint>

#include "fa_kernels.h"
#include "ptx.cuh"

namespace fa {

// freq (radians per position) -> turns per position, 64-bit fraction.
__device__ __forceinline__ unsigned long long turn_fraction(double freq) {
  double t = freq * 0.15915494309189533577;  // 1 / (2 pi)
  t -= floor(t);
  return __double2ull_rn(t * 18446744073709551616.0);  // t <= 1 - 2^-53: below 2^64
}

__device__ __forceinline__ void turn_sincos(unsigned long long fraction, long long position, float sign, float mscale,
                                            float& s, float& c) {
  const unsigned long long f = fraction * static_cast<unsigned long long>(position);
  // nearest multiple of 2^-32 of a turn, as half turns in [-1, 1)
  const int top = static_cast<int>(static_cast<unsigned>((f + 0x80000000ull) >> 32));
  sincospif(static_cast<float>(top) * 4.656612873077392578125e-10f, &s, &c);  // 2^-31
  s *= sign * mscale;
  c *= mscale;
}

// Sequence and place of a token; the 64-bit division, some ten times the
// 32-bit one, only where the number needs it.
__device__ __forceinline__ void token_at(long long token, const RotaryParams& p, int& z, int& n) {
  if (token <= 0xffffffffLL) {
    const unsigned t = static_cast<unsigned>(token), N = static_cast<unsigned>(p.N);
    z = static_cast<int>(t / N);
    n = static_cast<int>(t % N);
  } else {
    z = static_cast<int>(token / p.N);
    n = static_cast<int>(token % p.N);
  }
}

// Pointers of head row `hh` (over all sides) of token (z, n); false: nothing
// to write.
__device__ __forceinline__ bool rotary_row(const RotaryParams& p, int hh, int z, int n, long long slot,
                                           const uint16_t*& src, uint16_t*& dst, bool& turn) {
  int s = 0;
  if (hh >= p.side[0].heads) {
    hh -= p.side[0].heads;
    s = 1;
    if (hh >= p.side[1].heads) {
      hh -= p.side[1].heads;
      s = 2;
    }
  }
  const RotarySide& d = p.side[s];
  turn = d.turn != 0;
  src = d.in + z * d.in_z + hh * d.in_h + n * d.in_n;
  if (d.mode == 1) {
    dst = d.out + slot * d.out_n + hh * d.out_h;
    return slot >= 0 && slot < p.cache_rows;
  }
  dst = d.out + z * d.out_z + hh * d.out_h + n * d.out_n;
  return true;
}

// 16-byte rows: `rot` a multiple of 16, every row 16-byte aligned.
template <bool BF, bool IL, int D>
__global__ void __launch_bounds__(128) fa_rotary_kernel(const RotaryParams p) {
  constexpr int LANES = D / 16;           // threads per token
  constexpr int TOKENS = 128 / LANES;     // tokens per block
  __shared__ unsigned long long fraction[D / 2];
  static_assert(D / 2 <= 128, "one thread per pair");
  if (static_cast<int>(threadIdx.x) < p.rot / 2) fraction[threadIdx.x] = turn_fraction(__ldg(p.freqs + threadIdx.x));
  __syncthreads();
  const int tl = threadIdx.x / LANES, c = threadIdx.x % LANES;
  const long long token = static_cast<long long>(blockIdx.x) * TOKENS + tl;
  if (token >= static_cast<long long>(p.Z) * p.N) return;
  int z, n;
  token_at(token, p, z, n);
  const bool turns = c < p.rot / 16;
  // this thread's two 8-value chunks of a row
  const int a0 = !turns || IL ? 16 * c : 8 * c;
  const int a1 = !turns || IL ? a0 + 8 : a0 + p.rot / 2;
  float sn[8], cs[8];
  if (turns) {
    const long long pos = __ldg(p.positions + z * p.pos_z + n);
#pragma unroll
    for (int e = 0; e < 8; ++e) turn_sincos(fraction[8 * c + e], pos, p.sign, p.mscale, sn[e], cs[e]);
  }
  const long long slot = p.slots != nullptr ? __ldg(p.slots + token) : 0;
  const int h_end = min(p.heads, (static_cast<int>(blockIdx.y) + 1) * p.heads_per_block);
  constexpr int U = 4;
  for (int h0 = blockIdx.y * p.heads_per_block; h0 < h_end; h0 += U) {
    uint4 x0[U], x1[U];
    uint16_t* dst[U];
    bool live[U], turn[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint16_t* src;
      live[u] = h0 + u < h_end && rotary_row(p, h0 + u, z, n, slot, src, dst[u], turn[u]);
      if (live[u]) {
        x0[u] = *reinterpret_cast<const uint4*>(src + a0);
        x1[u] = *reinterpret_cast<const uint4*>(src + a1);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!live[u]) continue;
      if (turns && turn[u]) {
        uint32_t w0[4] = {x0[u].x, x0[u].y, x0[u].z, x0[u].w}, w1[4] = {x1[u].x, x1[u].y, x1[u].z, x1[u].w};
        if constexpr (IL) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 v = unpack2<BF>(w0[e]), w = unpack2<BF>(w1[e]);
            w0[e] = pack2<BF>(v.x * cs[e] - v.y * sn[e], v.y * cs[e] + v.x * sn[e]);
            w1[e] = pack2<BF>(w.x * cs[4 + e] - w.y * sn[4 + e], w.y * cs[4 + e] + w.x * sn[4 + e]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 v = unpack2<BF>(w0[e]), w = unpack2<BF>(w1[e]);
            w0[e] = pack2<BF>(v.x * cs[2 * e] - w.x * sn[2 * e], v.y * cs[2 * e + 1] - w.y * sn[2 * e + 1]);
            w1[e] = pack2<BF>(w.x * cs[2 * e] + v.x * sn[2 * e], w.y * cs[2 * e + 1] + v.y * sn[2 * e + 1]);
          }
        }
        x0[u] = make_uint4(w0[0], w0[1], w0[2], w0[3]);
        x1[u] = make_uint4(w1[0], w1[1], w1[2], w1[3]);
      }
      *reinterpret_cast<uint4*>(dst[u] + a0) = x0[u];
      *reinterpret_cast<uint4*>(dst[u] + a1) = x1[u];
    }
  }
}

// Any even `rot` and any alignment: one thread per pair (or two copied
// values) of a token.
template <bool BF, bool IL>
__global__ void __launch_bounds__(128) fa_rotary_any_kernel(const RotaryParams p) {
  const int lanes = p.D / 2;
  const long long total = static_cast<long long>(p.Z) * p.N * lanes;
  const long long x = static_cast<long long>(blockIdx.x) * 128 + threadIdx.x;
  if (x >= total) return;
  const long long token = x / lanes;
  const int c = static_cast<int>(x - token * lanes);
  int z, n;
  token_at(token, p, z, n);
  const bool turns = c < p.rot / 2;
  const int a0 = !turns || IL ? 2 * c : c;
  const int a1 = !turns || IL ? a0 + 1 : c + p.rot / 2;
  float sn = 0.f, cs = 1.f;
  if (turns)
    turn_sincos(turn_fraction(__ldg(p.freqs + c)), __ldg(p.positions + z * p.pos_z + n), p.sign, p.mscale, sn, cs);
  const long long slot = p.slots != nullptr ? __ldg(p.slots + token) : 0;
  const int h_end = min(p.heads, (static_cast<int>(blockIdx.y) + 1) * p.heads_per_block);
#pragma unroll 4
  for (int h = blockIdx.y * p.heads_per_block; h < h_end; ++h) {
    const uint16_t* src;
    uint16_t* dst;
    bool turn;
    if (!rotary_row(p, h, z, n, slot, src, dst, turn)) continue;
    const uint16_t v = src[a0], w = src[a1];
    uint32_t r = static_cast<uint32_t>(v) | static_cast<uint32_t>(w) << 16;
    if (turns && turn) {
      const float2 f = unpack2<BF>(r);
      r = pack2<BF>(f.x * cs - f.y * sn, f.y * cs + f.x * sn);
    }
    dst[a0] = static_cast<uint16_t>(r & 0xffffu);
    dst[a1] = static_cast<uint16_t>(r >> 16);
  }
}

int launch_rotary(const RotaryParams& prm, bool bf16, bool interleaved, bool wide, int num_sms, cudaStream_t stream) {
  RotaryParams p = prm;
  const int per_block = wide ? 128 / (p.D / 16) : 1;
  const long long tokens = static_cast<long long>(p.Z) * p.N;
  const long long blocks = wide ? (tokens + per_block - 1) / per_block : (tokens * (p.D / 2) + 127) / 128;
  if (blocks > 0x7fffffffLL) return -1;
  // heads dealt over the grid's y until there are about 8 blocks (1024
  // threads) per SM, at most one block per head
  long long groups = (8LL * num_sms + blocks - 1) / blocks;
  if (groups > p.heads) groups = p.heads;
  p.heads_per_block = static_cast<int>((p.heads + groups - 1) / groups);
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((p.heads + p.heads_per_block - 1) / p.heads_per_block));
  auto go = [&](auto kernel) { kernel<<<grid, 128, 0, stream>>>(p); };
  if (!wide) {
    if (bf16) interleaved ? go(fa_rotary_any_kernel<true, true>) : go(fa_rotary_any_kernel<true, false>);
    else interleaved ? go(fa_rotary_any_kernel<false, true>) : go(fa_rotary_any_kernel<false, false>);
  } else if (p.D == 64) {
    if (bf16) interleaved ? go(fa_rotary_kernel<true, true, 64>) : go(fa_rotary_kernel<true, false, 64>);
    else interleaved ? go(fa_rotary_kernel<false, true, 64>) : go(fa_rotary_kernel<false, false, 64>);
  } else if (p.D == 128) {
    if (bf16) interleaved ? go(fa_rotary_kernel<true, true, 128>) : go(fa_rotary_kernel<true, false, 128>);
    else interleaved ? go(fa_rotary_kernel<false, true, 128>) : go(fa_rotary_kernel<false, false, 128>);
  } else {
    if (bf16) interleaved ? go(fa_rotary_kernel<true, true, 256>) : go(fa_rotary_kernel<true, false, 256>);
    else interleaved ? go(fa_rotary_kernel<false, true, 256>) : go(fa_rotary_kernel<false, false, 256>);
  }
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace fa
