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

// True in one lane of the warp, always the same one (the one that issues MMAs
// and their commits); the branch on it leaves the warp's values uniform.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Products of 128-row tiles in shared memory (128-byte swizzle, panels of 64
// columns).  Only the low word of an operand's descriptor (address and leading
// offset) changes from one MMA to the next, by a constant: the issuing thread
// adds, it does not build descriptors (building them took longer than the MMA:
// 125 cycles per 128 x 128 x 16 product instead of 64 to 80).
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);   // stride 1024, version 1, 128-byte swizzle
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t lead_bytes) {
  return (saddr >> 4) | ((lead_bytes >> 4) << 16);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %4};\n\tmov.b64 db, {%2, %4};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(kDescHigh), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %4};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b), "r"(idesc), "r"(kDescHigh), "r"(accumulate)
      : "memory");
}
// D = A B^T: both operands contracted over the head dimension.
template <int HD>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t sa, uint32_t sb) {
  const uint32_t a = desc_low(sa, 16), b = desc_low(sb, 16);
#pragma unroll
  for (int kk = 0; kk < HD / 16; ++kk) {
    const uint32_t off = (kk >> 2) * (128 * 128 / 16) + (kk & 3) * 2;
    mma_ss(d, a + off, b + off, idesc_bf16_f32(128, 128, 0, 0), kk > 0 ? 1u : 0u);
  }
}
// D (+)= A B: A bf16 in TMEM (128 values of a row as pairs; the second half
// starts `half` columns after the first), B's 128 rows contracted.
template <int HD>
__device__ __forceinline__ void mma_cols(uint32_t d, uint32_t ta, uint32_t half, uint32_t sb, bool accumulate) {
  const uint32_t b = desc_low(sb, 128 * 128);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    mma_ts(d, ta + (kk >> 2) * half + 8u * (kk & 3), b + kk * (2048 / 16), idesc_bf16_f32(128, HD, 0, 1),
           (accumulate || kk > 0) ? 1u : 0u);
}

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

// Writes zeros over the rows 32 w0 .. 32 w0 + 63 of a shared-memory tile (panels
// of 64 columns, 128 bytes a row) whose bit is not set, and makes them visible
// to MMAs and TMA (whole warp): eight lanes a row, the row's bits being known to
// all.
template <int HD>
__device__ __forceinline__ void zero_hidden_rows(uint8_t* tile, uint4 seen, int w0, int lane) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t hidden = ~(w0 + i == 0 ? seen.x : w0 + i == 1 ? seen.y : w0 + i == 2 ? seen.z : seen.w);
    while (hidden) {       // four rows a time, a group of eight lanes each
      uint32_t rest = hidden;
      for (int g = lane >> 3; g > 0 && rest; --g) rest &= rest - 1;
      if (rest) {
        uint8_t* row = tile + (32 * (w0 + i) + __ffs(rest) - 1) * 128 + (lane & 7) * 16;
#pragma unroll
        for (int p = 0; p < HD / 64; ++p)
          *reinterpret_cast<uint4*>(row + p * 128 * 128) = make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) hidden &= hidden - 1;
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// Writes 64 columns (from column c0) of the warp's 32 rows of a query tile (tile
// rows row0 ..) to a per-token tensor, bf16(o * by), through `stage` (4 KB of the
// warp's own, 1024-byte aligned, no longer read): as one TMA store of lane 0's
// next bulk group, or, where a warp's rows are not whole tokens, with stores of
// 128 bytes of four rows each instead of 16 bytes of 32.
__device__ __forceinline__ void store_rows64(const CrossArgs& a, const CrossTiles& t, const CUtensorMap* map,
                                             const View& v, const Work& w, uint8_t* stage, int row0, int c0,
                                             const uint32_t* o, float by, int lane) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    uint4 u;
    u.x = pack_bf16x2(__uint_as_float(o[8 * e + 0]) * by, __uint_as_float(o[8 * e + 1]) * by);
    u.y = pack_bf16x2(__uint_as_float(o[8 * e + 2]) * by, __uint_as_float(o[8 * e + 3]) * by);
    u.z = pack_bf16x2(__uint_as_float(o[8 * e + 4]) * by, __uint_as_float(o[8 * e + 5]) * by);
    u.w = pack_bf16x2(__uint_as_float(o[8 * e + 6]) * by, __uint_as_float(o[8 * e + 7]) * by);
    *reinterpret_cast<uint4*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) = u;
  }
  if (t.bulk_out) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && w.real) {
      tma_store_4d(map, smem_addr(stage), c0, w.h0, w.tok0 + (int)fdiv((uint32_t)row0, t.div_pack), w.b);
      bulk_commit();
    }
    return;
  }
  __syncwarp();
  __nv_bfloat16* base = reinterpret_cast<__nv_bfloat16*>(v.p) + w.b * v.b + c0 + (lane & 7) * 8;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (lane >> 3);
    const uint4 u = *reinterpret_cast<const uint4*>(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
    const int rt = (int)fdiv((uint32_t)(row0 + r), t.div_pack), n = w.tok0 + rt, h = w.h0 + row0 + r - rt * t.pack;
    if (w.real && rt < t.tokens && n < a.n_q) *reinterpret_cast<uint4*>(base + n * v.n + h * v.h) = u;
  }
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
