// Windows with sinks, backward: dK and dV of the key tiles whose query tiles
// were cut into a near and several far units, from the units' fp32 partial sums
// (SinkTile):
//   dv[key] = near + far 1 + far 2 + ...,  dk[key] = scale (the same sum),
// in that order whatever the launch, so results are the same bit for bit.
// A warp takes 128 values of a key's [dV | dK] row.  Bound by the partial rows
// it reads, which are few: 128 rows of a near unit, and only the sinks' rows of
// a far one.
#include "fa_kernels.h"
#include "ptx.cuh"

namespace fa {

template <bool BF>
__global__ void __launch_bounds__(256) fa_sink_join_kernel(const BwdParams prm, int D, int bm, int tiles) {
  const int per_row = 2 * D / 128;  // warps per key
  const long long w = static_cast<long long>(blockIdx.x) * 8 + threadIdx.x / 32;
  const long long item = w / per_row;
  const int col = static_cast<int>(w % per_row) * 128 + (threadIdx.x & 31) * 4;
  const int row = static_cast<int>(item % 128), j = static_cast<int>(item / 128 % tiles);
  const int kvh = static_cast<int>(item / 128 / tiles);
  if (kvh >= prm.heads / prm.group || j * 128 + row >= prm.Nk) return;
  const SinkTile t = bm == 64 ? sink_tile<64>(j, prm.rule.sinks, prm.rule.window, prm.Nq, prm.causal_off, prm.far_tiles)
                              : sink_tile<128>(j, prm.rule.sinks, prm.rule.window, prm.Nq, prm.causal_off, prm.far_tiles);
  if (t.far == 0) return;  // its one unit wrote dK and dV
  const int before = bm == 64 ? sink_far_before<64, int>(j, prm.rule.window, prm.Nq, prm.causal_off, prm.far_tiles)
                              : sink_far_before<128, int>(j, prm.rule.window, prm.Nq, prm.causal_off, prm.far_tiles);
  const long long at = 128LL * (j + before);  // (as the units count: sink_dkdv_unit)
  const float* src = prm.part + kvh * prm.part_floats + (at + row) * 2 * D + col;
  float4 s = *reinterpret_cast<const float4*>(src);
  if (row < t.rows) {
    src += 128LL * 2 * D;
#pragma unroll 4
    for (int f = 0; f < t.far; ++f) {
      const float4 x = *reinterpret_cast<const float4*>(src + static_cast<long long>(f) * t.rows * 2 * D);
      s.x += x.x;
      s.y += x.y;
      s.z += x.z;
      s.w += x.w;
    }
  }
  const bool dk = col >= D;
  const float mul = dk ? prm.scale : 1.f;
  // dK and dV leave in the inputs' 16 bits, rounded once from the fp32 sum
  const uint2 h = make_uint2(pack2<BF>(s.x * mul, s.y * mul), pack2<BF>(s.z * mul, s.w * mul));
  __half* out = dk ? prm.dk + (col - D) : prm.dv + col;
  *reinterpret_cast<uint2*>(out + (static_cast<size_t>(kvh) * prm.Nk + j * 128 + row) * D) = h;
}

int launch_sink_join(const BwdParams& prm, int D, bool bf16, cudaStream_t stream) {
  const int tiles = (prm.rule.sinks + 127) / 128;
  const long long warps = static_cast<long long>(prm.heads / prm.group) * tiles * 128 * (2 * D / 128);
  const long long blocks = (warps + 7) / 8;
  if (blocks > 0x7fffffffLL) return -1;
  const int bm = D == 256 ? 64 : 128;  // query rows per tile of the dK/dV kernel
  if (bf16) {
    fa_sink_join_kernel<true><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(prm, D, bm, tiles);
  } else {
    fa_sink_join_kernel<false><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(prm, D, bm, tiles);
  }
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace fa
