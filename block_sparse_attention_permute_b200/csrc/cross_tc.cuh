// cross_tc.cuh — what the tensor-core kernels of cross attention share: the
// register split, the walk over items and key tiles, the mask bits of a tile.
#pragma once
#include "cross.cuh"

namespace bsa {

constexpr int kThreads = 384;   // two warpgroups of row work, one of loads (warp 8) and MMAs (warp 9)
// Registers: the launch gives kRegsLaunch to each thread; the load/MMA
// warpgroup then drops to kRegsSmall and the warpgroups of row work rise to
// kRegsRows.  (216 and 72 spill in the MMA warp, 1 to 2% slower.)
constexpr int kRegsLaunch = 168, kRegsRows = 200, kRegsSmall = 104;
static_assert(2 * 128 * kRegsRows + 128 * kRegsSmall <= kThreads * kRegsLaunch, "register split exceeds the launch");
__device__ __forceinline__ void take_row_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsRows));
}
__device__ __forceinline__ void give_up_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsSmall));
}

// An item of the schedule: a K/V head of a batch element, a run of key steps, a
// pair of query tiles (or one).
struct Work {
  int b, hk, bh;      // batch element, K/V head, and both as one index
  int keys;           // keys of the batch element
  int i, split;       // place among the head's items, key split
  int kt, n;          // first key step, steps (of stream 0 where the streams halve them)
  int all;            // steps of both streams together where they halve them, else n
  bool halved;
  // Steps of stream x and the first of them.
  __device__ __forceinline__ int steps(int x) const { return halved && x ? all - n : n; }
  __device__ __forceinline__ int first(int x) const { return halved && x ? kt + n : kt; }
};

__device__ __forceinline__ Work decode(const CrossArgs& a, const CrossTiles& t, int it) {
  Work w;
  const int rest = (int)fdiv((uint32_t)it, t.div_items);
  w.i = it - rest * (int)t.div_items.d;
  w.bh = (int)fdiv((uint32_t)rest, t.div_splits);
  w.split = rest - w.bh * (int)t.div_splits.d;
  w.b = (int)fdiv((uint32_t)w.bh, t.div_hkv);
  w.hk = w.bh - w.b * a.heads_kv;
  w.keys = cross_keys(a, w.b);
  w.kt = w.split * a.split_len;
  w.all = max(0, min(a.split_len, (w.keys + t.step - 1) / t.step - w.kt));
  w.halved = !t.shared;
  w.n = w.halved ? (w.all + 1) >> 1 : w.all;
  return w;
}

// The query tile that an item gives to stream x.
struct RowTile {
  int h0, tok0;   // first head and token
  int at;         // place among all query tiles
  bool real;      // false: the padding tile of an odd pair
};
__device__ __forceinline__ RowTile row_tile(const CrossArgs& a, const CrossTiles& t, const Work& w, int x) {
  const int tile = t.shared ? 2 * w.i + x : w.i;
  const int sg = (int)fdiv((uint32_t)tile, t.div_tok);
  return {w.hk * a.group + sg * t.pack, (tile - sg * (int)t.div_tok.d) * t.tokens, w.bh * t.tiles + tile,
          tile < t.tiles};
}

// Walks the steps of the CTA's items, both streams in step.
struct Cursor {
  int it, s;
  Work w;
  __device__ __forceinline__ bool valid(const CrossTiles& t) const { return it < t.items; }
  __device__ __forceinline__ bool active(int x) const { return s < w.steps(x); }
  __device__ __forceinline__ int key_step(int x) const { return w.first(x) + s; }
  __device__ __forceinline__ void find(const CrossArgs& a, const CrossTiles& t) {
    for (; it < t.items; it += gridDim.x) {
      w = decode(a, t, it);
      if (w.n > 0) break;
    }
    s = 0;
  }
  __device__ __forceinline__ void start(const CrossArgs& a, const CrossTiles& t) {
    it = blockIdx.x;
    find(a, t);
  }
  __device__ __forceinline__ void advance(const CrossArgs& a, const CrossTiles& t) {
    if (++s == w.n) {
      it += gridDim.x;
      find(a, t);
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
    const uint32_t p = kk >> 2, c = (kk & 3) * 2;
    mma_ss(d, a + p * (128 * 128 / 16) + c, b + p * (128 * 128 / 16) + c, idesc_bf16_f32(128, 128, 0, 0),
           kk > 0 ? 1u : 0u);
  }
}
// D (+)= A B: A bf16 in TMEM (128 values of a row as pairs; the second half starts
// `half` columns after the first), B's 128 rows contracted.
template <int HD>
__device__ __forceinline__ void mma_cols(uint32_t d, uint32_t ta, uint32_t half, uint32_t sb, bool accumulate) {
  const uint32_t b = desc_low(sb, 128 * 128);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    mma_ts(d, ta + (kk >> 2) * half + 8u * (kk & 3), b + kk * (2048 / 16), idesc_bf16_f32(128, HD, 0, 1),
           (accumulate || kk > 0) ? 1u : 0u);
}

// Bit c: key j0 + c is attended (whole warp).
__device__ __forceinline__ uint32_t seen_word(const CrossArgs& a, int b, int j0, int keys, int lane) {
  const int j = j0 + lane;
  bool s = j < keys;
  if (s && a.key_mask) s = __ldg(a.key_mask + (long long)b * a.n_kv + j) != 0;
  return __ballot_sync(0xffffffffu, s);
}

// Writes zeros over the rows of a shared-memory tile (128 bytes a row in each of
// its panels of 64 columns) whose bit in `hidden` is set, and makes them visible
// to MMAs and TMA (whole warp): four rows a time, a group of eight lanes each.
template <int HD>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int panel, uint32_t hidden, int lane) {
  while (hidden) {
    uint32_t rest = hidden;
    for (int g = lane >> 3; g > 0 && rest; --g) rest &= rest - 1;
    if (rest) {
      uint8_t* row = tile + (__ffs(rest) - 1) * 128 + (lane & 7) * 16;
#pragma unroll
      for (int p = 0; p < HD / 64; ++p) *reinterpret_cast<uint4*>(row + p * panel) = make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) hidden &= hidden - 1;
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// Output rows go from registers to a per-token tensor through shared memory: 32
// rows of the warp's own, 64 columns (4 KB, 1024-byte aligned) at a time, as
// bf16(o * by) in the 128-byte swizzle ...
__device__ __forceinline__ void stage_rows64(uint8_t* stage, const uint32_t* o, float by, int lane) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    uint4 u;
    u.x = pack_bf16x2(__uint_as_float(o[8 * e + 0]) * by, __uint_as_float(o[8 * e + 1]) * by);
    u.y = pack_bf16x2(__uint_as_float(o[8 * e + 2]) * by, __uint_as_float(o[8 * e + 3]) * by);
    u.z = pack_bf16x2(__uint_as_float(o[8 * e + 4]) * by, __uint_as_float(o[8 * e + 5]) * by);
    u.w = pack_bf16x2(__uint_as_float(o[8 * e + 6]) * by, __uint_as_float(o[8 * e + 7]) * by);
    *reinterpret_cast<uint4*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) = u;
  }
}
// ... and from there (tile rows row0 .. row0 + 31, whole warp) by TMA, in lane
// 0's next bulk group, or, where a warp's rows are not whole tokens, with stores
// of 128 bytes of four rows each (after which the stage is no longer read).
template <int HD>
__device__ __forceinline__ void store_rows(const CrossArgs& a, const CrossTiles& t, const CUtensorMap* map,
                                           const View& v, int b, const RowTile& q, uint8_t* stage, int row0, int lane) {
  fence_proxy_async_smem();
  __syncwarp();
  if (t.bulk_out) {
    if (lane == 0 && q.real) {
      const int tok = q.tok0 + (int)fdiv((uint32_t)row0, t.div_pack);
#pragma unroll
      for (int c0 = 0; c0 < HD; c0 += 64) tma_store_4d(map, smem_addr(stage + c0 * 64), c0, q.h0, tok, b);
      bulk_commit();
    }
    return;
  }
  __nv_bfloat16* base = reinterpret_cast<__nv_bfloat16*>(v.p) + b * v.b + (lane & 7) * 8;
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (lane >> 3);
    const int rt = (int)fdiv((uint32_t)(row0 + r), t.div_pack), n = q.tok0 + rt, h = q.h0 + row0 + r - rt * t.pack;
    if (q.real && rt < t.tokens && n < a.n_q) {
#pragma unroll
      for (int c0 = 0; c0 < HD; c0 += 64)
        *reinterpret_cast<uint4*>(base + c0 + n * v.n + h * v.h) =
            *reinterpret_cast<const uint4*>(stage + c0 * 64 + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// Before the first launch on a device: refuses a build whose kernel does not get
// kRegsLaunch registers per thread (the register split assumes it), and sets the
// shared-memory size.
template <class K>
inline cudaError_t prepare_kernel(K kernel, int smem) {
  cudaFuncAttributes attr;
  cudaError_t e = cudaFuncGetAttributes(&attr, kernel);
  if (e != cudaSuccess) return e;
  if (attr.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

}  // namespace bsa
