// cross_tc.cuh — what the tensor-core kernels of cross attention share: the
// register split, the walk over items and key tiles, the mask bits of a tile.
#pragma once
#include "cross.cuh"

namespace bsa {

constexpr int kThreads = 384;   // two warpgroups of row work, one of loads (warp 8) and MMAs (warp 9)
// Registers: the launch gives kRegsLaunch to each thread; the load/MMA
// warpgroup then drops to SMALL and the warpgroups of row work rise to ROWS.
constexpr int kRegsLaunch = 168;
template <int ROWS, int SMALL>
struct RegSplit {
  static_assert(2 * 128 * ROWS + 128 * SMALL <= kThreads * kRegsLaunch, "register split exceeds the launch");
  static __device__ __forceinline__ void rows() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(ROWS)); }
  static __device__ __forceinline__ void small() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(SMALL)); }
};

// What an item gives to one stream.
struct Work {
  int b, hk, h0, tok0;   // batch element, K/V head, first head and token of the query tile
  int kt, n;             // key tiles kt .. kt + n - 1
  int split;             // index of its partial
  int row_tile;          // its place among all query tiles
  bool real;             // false: the padding tile of an odd pair
};

__device__ __forceinline__ Work decode(const CrossArgs& a, const CrossTiles& t, int it, int x) {
  Work w;
  const int rest = (int)fdiv((uint32_t)it, t.div_items), i = it - rest * (int)t.div_items.d;
  const int bh = (int)fdiv((uint32_t)rest, t.div_splits);
  w.split = rest - bh * (int)t.div_splits.d;
  w.b = (int)fdiv((uint32_t)bh, t.div_hkv);
  w.hk = bh - w.b * a.heads_kv;
  const int tile = t.shared ? 2 * i + x : i;
  const int sg = (int)fdiv((uint32_t)tile, t.div_tok), tt = tile - sg * (int)t.div_tok.d;
  w.real = tile < t.tiles;
  w.row_tile = bh * t.tiles + tile;
  w.h0 = w.hk * a.group + sg * t.pack;
  w.tok0 = tt * t.tokens;
  const int tiles = (cross_keys(a, w.b) + 127) >> 7;
  w.kt = w.split * a.split_len;
  w.n = max(0, min(a.split_len, tiles - w.kt));
  if (!t.shared) {
    const int first = (w.n + 1) >> 1;
    w.split = 2 * w.split + x;
    if (x) w.kt += first;
    w.n = x ? w.n - first : first;
  }
  return w;
}

// Walks the steps of one stream over the CTA's items.
struct Cursor {
  int it, s;
  Work w;
  __device__ __forceinline__ bool valid(const CrossTiles& t) const { return it < t.items; }
  __device__ __forceinline__ void find(const CrossArgs& a, const CrossTiles& t, int x) {
    for (; it < t.items; it += gridDim.x) {
      w = decode(a, t, it, x);
      if (w.n > 0) break;
    }
    s = 0;
  }
  __device__ __forceinline__ void start(const CrossArgs& a, const CrossTiles& t, int x) {
    it = blockIdx.x;
    find(a, t, x);
  }
  __device__ __forceinline__ void advance(const CrossArgs& a, const CrossTiles& t, int x) {
    if (++s == w.n) {
      it += gridDim.x;
      find(a, t, x);
    }
  }
};

// Bit c of word w: key j0 + 32 w + c is attended (whole warp).
__device__ __forceinline__ uint4 seen_bits(const CrossArgs& a, int b, int j0, int keys, int lane) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = j0 + 32 * i + lane;
    bool s = j < keys;
    if (s && a.key_mask) s = __ldg(a.key_mask + (long long)b * a.n_kv + j) != 0;
    w[i] = __ballot_sync(0xffffffffu, s);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Writes zeros over the rows of a shared-memory tile (panels of 64 columns, 128
// bytes a row) whose bit is not set, and makes them visible to MMAs and TMA
// (whole warp).
template <int HD>
__device__ __forceinline__ void zero_hidden_rows(uint8_t* tile, uint4 seen, int lane) {
  const uint32_t m4[4] = {seen.x, seen.y, seen.z, seen.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (!((m4[i] >> lane) & 1u)) {
      uint8_t* row = tile + (32 * i + lane) * 128;
#pragma unroll
      for (int p = 0; p < HD / 64; ++p)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          reinterpret_cast<uint4*>(row + p * 128 * 128)[e] = make_uint4(0u, 0u, 0u, 0u);
    }
  fence_proxy_async_smem();
  __syncwarp();
}

// Refuses to launch a build whose kernel does not get kRegsLaunch registers per
// thread (the register split assumes it), and sets the shared-memory size.
template <class K>
cudaError_t prepare_kernel(K kernel, int smem) {
  cudaFuncAttributes attr;
  cudaError_t e = cudaFuncGetAttributes(&attr, kernel);
  if (e != cudaSuccess) return e;
  if (attr.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

}  // namespace bsa
