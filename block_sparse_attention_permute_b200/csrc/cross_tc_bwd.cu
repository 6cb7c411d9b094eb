// cross_tc_bwd.cu — gradients of cross attention on the tensor cores (bf16).
//
// With S = Q K^T, P = exp(scale S - lse), dP = dO V^T, delta = rowsum(dO * O),
// dS = P * (dP - delta):  dQ = scale dS K, dK = scale dS^T Q, dV = P^T dO.
// P and dS are rounded to bf16 as operands, the type of the tensors they multiply
// (tcgen05 takes both operands in one 16-bit type); delta is read from the rounded O
// where the keys fill more than one tile.  Together 0.3% of a gradient in norm.
// Both kernels form S and dP anew (seven products in all where five would do):
// dQ sums over keys and dK, dV over query rows, and with the sum in TMEM each
// has a fixed order and needs no fp32 traffic through L2 or atomics.
//
// cross_tc_dq: two streams of query tiles per persistent CTA over the same key
// tiles, as in the forward; a thread owns a query row.  TMEM: S, then dP, then
// dS (bf16) of stream x at 128 x (P waits in registers), dQ at 256 + 128 x.
//   S0(0) S1(0) | dP0(0) dP1(0) dQ0(0) S0(1) dQ1(0) S1(1) | dP0(1) ...
// cross_tc_dkv: a CTA owns 128 keys and a run of query tiles; a thread owns a
// key and half of a tile's queries.  TMEM: S^T and P^T at 0, dP^T and dS^T at
// 128, dV at 256, dK at 384.
//   S(0) dP(0) | dV(0) S(1) dK(0) dP(1) | dV(1) S(2) dK(1) dP(2) | ...
// so that the row work on P runs beside dK and dP, and that on dS beside dV and
// the next S.
//
// Measured on B200, 32 760 queries x 512 keys x 12 heads of 128 (a product is 51.5
// GFLOP): row sums 36 us (203 MB, 5.6 TB/s), dQ 147 us (three products, 1050
// TFLOP/s), dK and dV 178 us (four, 1160 TFLOP/s), their reduction 10 us, each alone at
// 1.8 to 1.9 GHz; 430 us together in a sustained loop at the 1000 W cap.  Tensor pipe
// 52 and 56% busy: bound by the row work between two products (1600 cycles for P of
// a tile, 600 for dS), beside which the other products run.
#include "cross_tc.cuh"

namespace bsa {
namespace {


// Shared memory of cross_tc_dq.
template <int HD>
struct DqLayout {
  static constexpr int kTile = 128 * HD * 2;
  static constexpr int kQ = 0, kDo = 2 * kTile, kK = 4 * kTile, kV = 6 * kTile;   // 2 Q, 2 dO, 2 K slots, 1 V
  static constexpr int kBars = 7 * kTile;
  static constexpr int kQFull = 0, kQEmpty = 2, kOFull = 4, kOEmpty = 6, kKFull = 8, kKEmpty = 10, kVFull = 12,
                       kVEmpty = 13, kS = 14, kP = 16, kDp = 18, kDs = 20, kDq = 22, kFinal = 24, kKClean = 25,
                       kVClean = 27, kNumBars = 28;
  static constexpr int kTmemSlot = kBars + kNumBars * 8, kAbort = kTmemSlot + 4;
  static constexpr int kAlloc = kAbort + 4 + 1024;
};

// Shared memory of cross_tc_dkv.
template <int HD>
struct DkvLayout {
  static constexpr int kTile = 128 * HD * 2;
  static constexpr int kStages = HD == 128 ? 2 : 4;
  static constexpr int kK = 0, kV = kTile, kQ = 2 * kTile, kDo = kQ + kStages * kTile, kStat = kDo + kStages * kTile;
  static constexpr int kBars = kStat + kStages * 1024;
  static constexpr int kKv = 0, kQFull = 1, kQEmpty = kQFull + kStages, kOFull = kQEmpty + kStages,
                       kOEmpty = kOFull + kStages, kS = kOEmpty + kStages, kP = kS + 1, kDp = kP + 1, kDs = kDp + 1,
                       kFinal = kDs + 1, kNumBars = kFinal + 1;
  static constexpr int kTmemSlot = kBars + kNumBars * 8, kAbort = kTmemSlot + 4;
  static constexpr int kAlloc = kAbort + 4 + 1024;
};

template <int HD>
__device__ __forceinline__ void load_tile4(uint32_t dst, const CUtensorMap* map, int h, int n, int b, uint32_t bar) {
#pragma unroll
  for (int p = 0; p < HD / 64; ++p) tma_load_4d(dst + p * (128 * 128), map, 64 * p, h, n, b, bar);
}

// 32 fp32 values of TMEM, times `by`, to a row of bf16 or fp32.
__device__ __forceinline__ void store32(__nv_bfloat16* d, const uint32_t (&o)[32], float by) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint4 v;
    v.x = pack_bf16x2(__uint_as_float(o[8 * c + 0]) * by, __uint_as_float(o[8 * c + 1]) * by);
    v.y = pack_bf16x2(__uint_as_float(o[8 * c + 2]) * by, __uint_as_float(o[8 * c + 3]) * by);
    v.z = pack_bf16x2(__uint_as_float(o[8 * c + 4]) * by, __uint_as_float(o[8 * c + 5]) * by);
    v.w = pack_bf16x2(__uint_as_float(o[8 * c + 6]) * by, __uint_as_float(o[8 * c + 7]) * by);
    reinterpret_cast<uint4*>(d)[c] = v;
  }
}
__device__ __forceinline__ void store32(float* d, const uint32_t (&o)[32], float by) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    reinterpret_cast<float4*>(d)[c] =
        make_float4(__uint_as_float(o[4 * c]) * by, __uint_as_float(o[4 * c + 1]) * by,
                    __uint_as_float(o[4 * c + 2]) * by, __uint_as_float(o[4 * c + 3]) * by);
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    cross_tc_dq(const __grid_constant__ CrossArgs a, const __grid_constant__ CrossTiles t,
                const __grid_constant__ CrossMaps maps) {
  using L = DqLayout<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_addr(sm);
  auto bar = [&](int x) { return sb + L::kBars + 8u * (uint32_t)x; };
  volatile int* abort = reinterpret_cast<volatile int*>(sm + L::kAbort);
  const long long lim = t.wait_limit > 0 ? t.wait_limit : kWaitLimitDefault;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool cleaning = a.key_mask != nullptr || a.kv_len != nullptr;

  if (threadIdx.x == 0) {
    for (int x = 0; x < L::kNumBars; ++x)
      mbar_init(bar(x), (x >= L::kP && x < L::kP + 2) || (x >= L::kDs && x < L::kDs + 2) ||
                                (x >= L::kOEmpty && x < L::kOEmpty + 2)
                            ? 128u
                            : x >= L::kKClean ? 2u : 1u);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(sb + L::kTmemSlot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + L::kTmemSlot);

  if (warp >= 8) {
    give_up_registers();
    if (warp == 8 && lane == 0) {
      // ------------------------------------------------------------ loads
      int g = 0, kv = 0, nq[2] = {0, 0}, no[2] = {0, 0};   // steps, K/V copies, copies of each Q and dO buffer
      int nk = 0, nv = 0;
      auto load = [&](int empty, int full, int done, int at, const CUtensorMap* map, int h, int n, int b) {
        if (done > 0 && !mbar_wait(bar(empty), (done - 1) & 1, abort, lim)) return false;
        mbar_arrive_expect_tx(bar(full), L::kTile);
        load_tile4<HD>(sb + at, map, h, n, b, bar(full));
        return true;
      };
      Cursor c;
      for (c.start(a, t); c.valid(t); c.advance(a, t), ++g) {
        const Work& w = c.w;
        // the padding tile of an odd pair lies past the tokens and reads zeros
        const RowTile r0 = row_tile(a, t, w, 0), r1 = row_tile(a, t, w, 1);
        const int h1 = r1.real ? r1.h0 : 0, tok1 = r1.real ? r1.tok0 : a.n_q;
        if (++kv == t.hold_load && blockIdx.x == 0) break;      // test hook: a copy that never lands
        const int ks = g & 1;
        if (!load(L::kKEmpty + ks, L::kKFull + ks, g >> 1, L::kK + ks * L::kTile, &maps.k, w.hk * t.step_kh,
                  (w.kt + c.s) * 128, w.b * t.step_kb))
          break;
        ++nk;
        if (c.s == 0) {
          if (!load(L::kQEmpty, L::kQFull, nq[0], L::kQ, &maps.q, r0.h0 * t.step_qh, r0.tok0, w.b * t.step_qb)) break;
          ++nq[0];
          if (!load(L::kQEmpty + 1, L::kQFull + 1, nq[1], L::kQ + L::kTile, &maps.q, h1 * t.step_qh, tok1,
                    w.b * t.step_qb))
            break;
          ++nq[1];
        }
        if (++kv == t.hold_load && blockIdx.x == 0) break;
        if (!load(L::kVEmpty, L::kVFull, g, L::kV, &maps.v, w.hk * t.step_vh, (w.kt + c.s) * 128, w.b * t.step_vb)) break;
        ++nv;
        if (c.s == 0) {
          if (!load(L::kOEmpty, L::kOFull, no[0], L::kDo, &maps.d_o, r0.h0 * t.step_oh, r0.tok0, w.b * t.step_ob)) break;
          ++no[0];
          if (!load(L::kOEmpty + 1, L::kOFull + 1, no[1], L::kDo + L::kTile, &maps.d_o, h1 * t.step_oh, tok1,
                    w.b * t.step_ob))
            break;
          ++no[1];
        }
      }
      // No copy is left in flight, also after an abort: issued copies land.
      for (int x = 0; x < 2; ++x) {
        if (nq[x] > 0) mbar_wait_drain(bar(L::kQFull + x), (nq[x] - 1) & 1, lim);
        if (no[x] > 0) mbar_wait_drain(bar(L::kOFull + x), (no[x] - 1) & 1, lim);
        if (nk > x) mbar_wait_drain(bar(L::kKFull + x), ((nk - 1 - x) >> 1) & 1, lim);
      }
      if (nv > 0) mbar_wait_drain(bar(L::kVFull), (nv - 1) & 1, lim);
    } else if (warp == 9) {
      // ------------------------------------------------------------ MMAs (the whole warp waits, one lane issues)
      auto wait = [&](int b, int phase) {
        return __all_sync(0xffffffffu, mbar_wait(bar(b), phase & 1, abort, lim)) != 0;
      };
      int items = 0;
      // S of both streams for step g (x = 0 also takes the K tile)
      auto score = [&](const Cursor& c, int g, int x) -> bool {
        const int ks = g & 1;
        if (c.s == 0 && !wait(L::kQFull + x, items)) return false;
        if (x == 0) {
          if (!wait((cleaning ? L::kKClean : L::kKFull) + ks, g >> 1)) return false;
        }
        tc_fence_after();
        if (elect_one()) {
          mma_rows<HD>(tmem + 128u * x, sb + L::kQ + x * L::kTile, sb + L::kK + ks * L::kTile);
          tc_commit(bar(L::kS + x));
          if (c.s == c.w.n - 1) tc_commit(bar(L::kQEmpty + x));
        }
        __syncwarp();
        return true;
      };
      Cursor c;
      c.start(a, t);
      bool ok = true;
      if (c.valid(t)) ok = score(c, 0, 0) && score(c, 0, 1);
      for (int g = 0; ok && c.valid(t); ++g) {
        const bool last = c.s == c.w.n - 1;
#pragma unroll
        for (int x = 0; x < 2 && ok; ++x) {
          if (c.s == 0) ok = wait(L::kOFull + x, items);
          if (ok && x == 0) ok = wait(cleaning ? L::kVClean : L::kVFull, g);
          if (ok) ok = wait(L::kP + x, g);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            mma_rows<HD>(tmem + 128u * x, sb + L::kDo + x * L::kTile, sb + L::kV);
            tc_commit(bar(L::kDp + x));
            if (x == 1) tc_commit(bar(L::kVEmpty));
          }
          __syncwarp();
        }
        if (!ok) break;
        Cursor next = c;
        next.advance(a, t);
        if (last) ++items;      // Q buffers of the next item
#pragma unroll
        for (int x = 0; x < 2 && ok; ++x) {
          ok = wait(L::kDs + x, g);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            mma_cols<HD>(tmem + 256u + 128u * x, tmem + 128u * x, 32u, sb + L::kK + (g & 1) * L::kTile, c.s > 0);
            if (last) tc_commit(bar(L::kDq + x));
            if (x == 1) tc_commit(bar(L::kKEmpty + (g & 1)));
          }
          __syncwarp();
          if (next.valid(t)) ok = score(next, g + 1, x);
        }
        c = next;
      }
      // Every MMA issued is complete before TMEM is released, also after an abort.
      if (elect_one()) tc_commit(bar(L::kFinal));
      mbar_wait_drain(bar(L::kFinal), 0, lim);
    } else if (warp >= 10 && cleaning) {
      // ------------------------------------------------------------ cleaning
      // What K and V hold at keys that are not attended must not enter, not even
      // times 0: warps 10 and 11 write zeros over those rows, 64 rows each.
      Cursor c;
      int g = 0;
      for (c.start(a, t); c.valid(t); c.advance(a, t), ++g) {
        const int j0 = (c.w.kt + c.s) * 128 + 64 * (warp - 10), ks = g & 1;
        const uint32_t hidden0 = ~seen_word(a, c.w.b, j0, c.w.keys, lane), hidden1 = ~seen_word(a, c.w.b, j0 + 32, c.w.keys, lane);
        auto clean = [&](uint8_t* tile) {
          tile += 64 * (warp - 10) * 128;
          if (hidden0) zero_rows<HD>(tile, 128 * 128, hidden0, lane);
          if (hidden1) zero_rows<HD>(tile + 32 * 128, 128 * 128, hidden1, lane);
        };
        if (!__all_sync(0xffffffffu, mbar_wait(bar(L::kKFull + ks), (g >> 1) & 1, abort, lim))) break;
        clean(sm + L::kK + ks * L::kTile);
        if (lane == 0) mbar_arrive(bar(L::kKClean + ks));
        if (!__all_sync(0xffffffffu, mbar_wait(bar(L::kVFull), g & 1, abort, lim))) break;
        clean(sm + L::kV);
        if (lane == 0) mbar_arrive(bar(L::kVClean));
      }
    }
  } else {
    // ------------------------------------------------------------ rows
    take_row_registers();
    const int x = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + 128u * x + lane_off, tQ = tmem + 256u + 128u * x + lane_off;
    const int rt = (int)fdiv((uint32_t)r, t.div_pack), rg = r - rt * t.pack;
    const long long rows = cross_rows(a);
    const float2 sl2 = make_float2(a.scale_log2, a.scale_log2);
    int g = 0, items = 0;
    bool ok = true;
    auto wait = [&](int b, int phase) {
      return __all_sync(0xffffffffu, mbar_wait(bar(b), phase & 1, abort, lim)) != 0;
    };
    for (int it = blockIdx.x; it < t.items && ok; it += gridDim.x) {
      const Work w = decode(a, t, it);
      const RowTile q = row_tile(a, t, w, x);
      float nl = -INFINITY, nd = 0.f;     // -lse (log2 units) and -delta of the row
      if (q.real) {
        nl = __ldg(a.stats + (long long)q.at * 256 + r);
        nd = __ldg(a.stats + (long long)q.at * 256 + 128 + r);
      }
      const float2 nl2 = make_float2(nl, nl);
      const bool one = one_key(a, w.b, w.keys);
      for (int s = 0; s < w.n; ++s, ++g) {
        const int j0 = (w.kt + s) * 128;
        const bool partial = a.key_mask != nullptr || j0 + 128 > w.keys;
        uint32_t w4[4];
        if (partial) {
#pragma unroll
          for (int i = 0; i < 4; ++i) w4[i] = seen_word(a, w.b, j0 + 32 * i, w.keys, lane);
        }
        if (!wait(L::kS + x, g)) { ok = false; break; }
        tc_fence_after();
        uint32_t p[128];
        TMEM_LD32(tS + 0, (p + 0));
        TMEM_LD32(tS + 32, (p + 32));
        TMEM_LD32(tS + 64, (p + 64));
        TMEM_LD32(tS + 96, (p + 96));
        TMEM_LD_WAIT((p + 0));
        TMEM_LD_WAIT((p + 32));
        TMEM_LD_WAIT((p + 64));
        TMEM_LD_WAIT((p + 96));
        // S is in registers: dP may take its place
        tc_fence_before();
        mbar_arrive(bar(L::kP + x));
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          const float2 e = fma2(make_float2(__uint_as_float(p[2 * c]), __uint_as_float(p[2 * c + 1])), sl2, nl2);
          p[2 * c] = __float_as_uint(fast_ex2(e.x));
          p[2 * c + 1] = __float_as_uint(fast_ex2(e.y));
        }
        if (partial) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (w4[i] == 0xffffffffu) continue;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!((w4[i] >> c) & 1u)) p[32 * i + c] = 0u;
          }
        }
        if (!wait(L::kDp + x, g)) { ok = false; break; }
        tc_fence_after();
        if (w.keys <= 128) {
          // All keys are here, so delta is the sum of P dP in fp32, not that of dO
          // with the rounded O: with few keys dP - delta cancels, and the rounding
          // of O was the largest error of dQ and dK (0.6% with two keys, else 0.25).
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            uint32_t d[32];
            TMEM_LD32(tS + 32 * y, d);
            TMEM_LD_WAIT(d);
#pragma unroll
            for (int c = 0; c < 16; ++c)
              sum = fma2(make_float2(__uint_as_float(p[32 * y + 2 * c]), __uint_as_float(p[32 * y + 2 * c + 1])),
                         make_float2(__uint_as_float(d[2 * c]), __uint_as_float(d[2 * c + 1])), sum);
          }
          nd = -(sum.x + sum.y);
          if (q.real) a.stats[(long long)q.at * 256 + 128 + r] = nd;     // for dK
        }
        if (one) {                        // dS = 0; a NaN stays one
#pragma unroll
          for (int c = 0; c < 128; ++c) p[c] = __float_as_uint(__uint_as_float(p[c]) * 0.f);
        }
        const float2 nd2 = make_float2(nd, nd);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[32];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            uint32_t d[32];
            TMEM_LD32(tS + 64 * h + 32 * y, d);
            TMEM_LD_WAIT(d);
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const int e = 64 * h + 32 * y + 2 * c;
              const float2 v = mul2(make_float2(__uint_as_float(p[e]), __uint_as_float(p[e + 1])),
                                    add2(make_float2(__uint_as_float(d[2 * c]), __uint_as_float(d[2 * c + 1])), nd2));
              pk[16 * y + c] = pack_bf16x2(v.x, v.y);
            }
          }
          TMEM_ST32(tS + 32 * h, pk);     // columns that this row has read
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar(L::kDs + x));
      }
      if (!ok) break;
      if (w.n > 0) {
        if (!wait(L::kDq + x, items)) { ok = false; break; }
        tc_fence_after();
        ++items;
      }
      const int n = q.tok0 + rt, h = q.h0 + rg;
      const bool row = q.real && n < a.n_q;
      const long long at = ((long long)w.b * a.heads + h) * a.n_q + n;
      if (a.splits > 1 || w.n == 0) {
#pragma unroll 1
        for (int c0 = 0; c0 < HD; c0 += 32) {
          uint32_t o[32];
          if (w.n > 0) {
            TMEM_LD32(tQ + c0, o);
            TMEM_LD_WAIT(o);
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = 0u;
          }
          if (row && a.splits > 1) store32(a.part_o + (w.split * rows + at) * HD + c0, o, a.scale);
          if (row && a.splits == 1)
            store32(reinterpret_cast<__nv_bfloat16*>(a.dq.p) + w.b * a.dq.b + n * a.dq.n + h * a.dq.h + c0, o, a.scale);
        }
      } else {
        // every MMA that reads the stream's dO is done: its place serves the
        // stores, and only then takes the next item's
        uint8_t* stage = sm + L::kDo + x * L::kTile + (warp & 3) * (L::kTile / 4);
#pragma unroll 1
        for (int c0 = 0; c0 < HD; c0 += 64) {
          uint32_t o[64];
          TMEM_LD32(tQ + c0, (o + 0));
          TMEM_LD32(tQ + c0 + 32, (o + 32));
          TMEM_LD_WAIT((o + 0));
          TMEM_LD_WAIT((o + 32));
          stage_rows64(stage + c0 * 64, o, a.scale, lane);
        }
        store_rows<HD>(a, t, &maps.out, a.dq, w.b, q, stage, (warp & 3) * 32, lane);
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
      }
      if (w.n > 0) {
        fence_proxy_async_smem();
        mbar_arrive(bar(L::kOEmpty + x));
      }
      tc_fence_before();
    }
    if (lane == 0) bulk_wait();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort) atomicCAS(a.status, 0, (int)BSA_ERR_TIMEOUT);
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    cross_tc_dkv(const __grid_constant__ CrossArgs a, const __grid_constant__ CrossTiles t,
                 const __grid_constant__ CrossMaps maps) {
  using L = DkvLayout<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_addr(sm);
  auto bar = [&](int x) { return sb + L::kBars + 8u * (uint32_t)x; };
  volatile int* abort = reinterpret_cast<volatile int*>(sm + L::kAbort);
  const long long lim = t.wait_limit > 0 ? t.wait_limit : kWaitLimitDefault;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // The CTA's keys and its run of query tiles; the runs of one key tile and the
  // key tiles of one head are neighbours.
  const int key_tiles = (a.n_kv + 127) >> 7;
  const int bh = blockIdx.x / (key_tiles * a.splits), rest = blockIdx.x - bh * key_tiles * a.splits;
  const int split = rest / key_tiles, j0 = (rest - split * key_tiles) * 128;
  const int b = bh / a.heads_kv, hk = bh - b * a.heads_kv;
  const int keys = cross_keys(a, b);
  const int t0 = split * a.split_len, n = j0 < keys ? min(a.split_len, t.tiles - t0) : 0;

  if (threadIdx.x == 0) {
    for (int x = 0; x < L::kNumBars; ++x) mbar_init(bar(x), x == L::kP || x == L::kDs ? 256u : 1u);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(sb + L::kTmemSlot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + L::kTmemSlot);
  const uint32_t tS = tmem, tD = tmem + 128, tV = tmem + 256, tK = tmem + 384;

  if (warp >= 8) {
    give_up_registers();
    if (warp == 8 && lane == 0 && n > 0) {
      // ------------------------------------------------------------ loads
      mbar_arrive_expect_tx(bar(L::kKv), 2 * L::kTile);
      load_tile4<HD>(sb + L::kK, &maps.k, hk * t.step_kh, j0, b * t.step_kb, bar(L::kKv));
      load_tile4<HD>(sb + L::kV, &maps.v, hk * t.step_vh, j0, b * t.step_vb, bar(L::kKv));
      int nq = 0, no = 0;
      for (int i = 0; i < n; ++i) {
        const int st = i % L::kStages, use = i / L::kStages, tile = t0 + i;
        const int sg = (int)fdiv((uint32_t)tile, t.div_tok), tok = (tile - sg * (int)t.div_tok.d) * t.tokens;
        const int h = hk * a.group + sg * t.pack;
        if (use > 0 && !mbar_wait(bar(L::kQEmpty + st), (use - 1) & 1, abort, lim)) break;
        mbar_arrive_expect_tx(bar(L::kQFull + st), L::kTile + 1024);
        load_tile4<HD>(sb + L::kQ + st * L::kTile, &maps.q, h * t.step_qh, tok, b * t.step_qb, bar(L::kQFull + st));
        bulk_load(sb + L::kStat + st * 1024, a.stats + ((long long)bh * t.tiles + tile) * 256, 1024, bar(L::kQFull + st));
        ++nq;
        if (use > 0 && !mbar_wait(bar(L::kOEmpty + st), (use - 1) & 1, abort, lim)) break;
        mbar_arrive_expect_tx(bar(L::kOFull + st), L::kTile);
        load_tile4<HD>(sb + L::kDo + st * L::kTile, &maps.d_o, h * t.step_oh, tok, b * t.step_ob, bar(L::kOFull + st));
        ++no;
      }
      // No copy is left in flight, also after an abort: issued copies land.
      mbar_wait_drain(bar(L::kKv), 0, lim);
      for (int i = nq > L::kStages ? nq - L::kStages : 0; i < nq; ++i)
        mbar_wait_drain(bar(L::kQFull + i % L::kStages), (i / L::kStages) & 1, lim);
      for (int i = no > L::kStages ? no - L::kStages : 0; i < no; ++i)
        mbar_wait_drain(bar(L::kOFull + i % L::kStages), (i / L::kStages) & 1, lim);
    } else if (warp == 9 && n > 0) {
      // ------------------------------------------------------------ MMAs (the whole warp waits, one lane issues)
      auto wait = [&](int x, int phase) {
        const bool ok = __all_sync(0xffffffffu, mbar_wait(bar(x), phase & 1, abort, lim)) != 0;
        tc_fence_after();
        return ok;
      };
      auto scores = [&](int i) {      // S^T of query tile i
        const int st = i % L::kStages;
        if (!wait(L::kQFull + st, i / L::kStages)) return false;
        if (elect_one()) {
          mma_rows<HD>(tS, sb + L::kK, sb + L::kQ + st * L::kTile);
          tc_commit(bar(L::kS));
        }
        __syncwarp();
        return true;
      };
      auto slopes = [&](int i) {      // dP^T of query tile i
        const int st = i % L::kStages;
        if (!wait(L::kOFull + st, i / L::kStages)) return false;
        if (elect_one()) {
          mma_rows<HD>(tD, sb + L::kV, sb + L::kDo + st * L::kTile);
          tc_commit(bar(L::kDp));
        }
        __syncwarp();
        return true;
      };
      bool ok = wait(L::kKv, 0) && scores(0) && slopes(0);
      for (int i = 0; ok && i < n; ++i) {
        const int st = i % L::kStages;
        if (!wait(L::kP, i)) break;
        if (elect_one()) {
          mma_cols<HD>(tV, tS, 64u, sb + L::kDo + st * L::kTile, i > 0);
          tc_commit(bar(L::kOEmpty + st));
        }
        __syncwarp();
        if (i + 1 < n && !scores(i + 1)) break;
        if (!wait(L::kDs, i)) break;
        if (elect_one()) {
          mma_cols<HD>(tK, tD, 64u, sb + L::kQ + st * L::kTile, i > 0);
          tc_commit(bar(L::kQEmpty + st));
        }
        __syncwarp();
        if (i + 1 < n && !slopes(i + 1)) break;
      }
      // The row threads read dK and dV after this; every MMA issued is complete
      // before TMEM is released, also after an abort.
      if (elect_one()) tc_commit(bar(L::kFinal));
      mbar_wait_drain(bar(L::kFinal), 0, lim);
    }
  } else {
    // ------------------------------------------------------------ keys
    take_row_registers();
    const int x = warp >> 2, r = (warp & 3) * 32 + lane, j = j0 + r;   // half of the queries, key
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    bool seen = j < keys;
    if (seen && a.key_mask) seen = __ldg(a.key_mask + (long long)b * a.n_kv + j) != 0;
    const bool one = one_key(a, b, keys);
    const float2 sl2 = make_float2(a.scale_log2, a.scale_log2);
    bool ok = true;
    auto wait = [&](int y, int phase) {
      return __all_sync(0xffffffffu, mbar_wait(bar(y), phase & 1, abort, lim)) != 0;
    };
    for (int i = 0; i < n; ++i) {
      const int st = i % L::kStages;
      // -lse and -delta of the thread's 64 queries (the wait is for their copy).
      // -lse is read ahead of S: beside the MMAs' operands shared memory is slow
      // (350 cycles of the step).
      if (!(ok = wait(L::kQFull + st, i / L::kStages))) break;
      const float4* nl = reinterpret_cast<const float4*>(sm + L::kStat + st * 1024) + 16 * x;
      const float4* nd = nl + 32;
      float4 lse[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) lse[c] = nl[c];
      if (!(ok = wait(L::kS, i))) break;
      tc_fence_after();
      uint32_t p[64], pk[32];
      TMEM_LD32(tS + lane_off + 64 * x, (p + 0));
      TMEM_LD32(tS + lane_off + 64 * x + 32, (p + 32));
      TMEM_LD_WAIT((p + 0));
      TMEM_LD_WAIT((p + 32));
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const float4 l = lse[c];
        const float2 e0 = fma2(make_float2(__uint_as_float(p[4 * c]), __uint_as_float(p[4 * c + 1])), sl2,
                               make_float2(l.x, l.y));
        const float2 e1 = fma2(make_float2(__uint_as_float(p[4 * c + 2]), __uint_as_float(p[4 * c + 3])), sl2,
                               make_float2(l.z, l.w));
        p[4 * c] = __float_as_uint(fast_ex2(e0.x));
        p[4 * c + 1] = __float_as_uint(fast_ex2(e0.y));
        p[4 * c + 2] = __float_as_uint(fast_ex2(e1.x));
        p[4 * c + 3] = __float_as_uint(fast_ex2(e1.y));
      }
      if (!seen) {
#pragma unroll
        for (int c = 0; c < 64; ++c) p[c] = 0u;
      }
#pragma unroll
      for (int c = 0; c < 32; ++c) pk[c] = pack_bf16x2(__uint_as_float(p[2 * c]), __uint_as_float(p[2 * c + 1]));
      TMEM_ST32(tS + lane_off + 64 * x, pk);     // over columns that this thread has read
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(bar(L::kP));
      if (one) {                          // dS = 0; a NaN stays one
#pragma unroll
        for (int c = 0; c < 64; ++c) p[c] = __float_as_uint(__uint_as_float(p[c]) * 0.f);
      }
      if (!(ok = wait(L::kDp, i))) break;
      tc_fence_after();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t d[32];
        TMEM_LD32(tD + lane_off + 64 * x + 32 * h, d);
        TMEM_LD_WAIT(d);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float4 l = nd[8 * h + c];
          const int e = 32 * h + 4 * c;
          const float2 v0 = mul2(make_float2(__uint_as_float(p[e]), __uint_as_float(p[e + 1])),
                                 add2(make_float2(__uint_as_float(d[4 * c]), __uint_as_float(d[4 * c + 1])),
                                      make_float2(l.x, l.y)));
          const float2 v1 = mul2(make_float2(__uint_as_float(p[e + 2]), __uint_as_float(p[e + 3])),
                                 add2(make_float2(__uint_as_float(d[4 * c + 2]), __uint_as_float(d[4 * c + 3])),
                                      make_float2(l.z, l.w)));
          pk[16 * h + 2 * c] = pack_bf16x2(v0.x, v0.y);
          pk[16 * h + 2 * c + 1] = pack_bf16x2(v1.x, v1.y);
        }
      }
      if (!seen) {
#pragma unroll
        for (int c = 0; c < 32; ++c) pk[c] = 0u;
      }
      TMEM_ST32(tD + lane_off + 64 * x, pk);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(bar(L::kDs));
    }
    if (n > 0 && ok) {
      ok = wait(L::kFinal, 0);
      tc_fence_after();
    }
    // Stream x writes half of the columns of dV and dK (head dimension 64: one of
    // the two); a key that is not attended gets zeros.
    if (ok && n > 0 && a.splits == 1 && a.slot_of == nullptr) {
      // through the places of K and V, which nothing reads any more, in runs of 128
      // bytes (with few query rows this is most of a CTA's time)
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        if (HD == 64 && which != x) continue;
        const int c0 = HD == 64 ? 0 : 64 * x;
        uint32_t o[64];
        TMEM_LD32((which ? tV : tK) + lane_off + c0, (o + 0));
        TMEM_LD32((which ? tV : tK) + lane_off + c0 + 32, (o + 32));
        TMEM_LD_WAIT((o + 0));
        TMEM_LD_WAIT((o + 32));
        if (!seen) {
#pragma unroll
          for (int c = 0; c < 64; ++c) o[c] = 0u;
        }
        uint8_t* stage = sm + (which ? L::kV : L::kK) + (HD == 64 ? warp & 3 : warp) * 4096;
        stage_rows64(stage, o, which ? 1.0f : a.scale, lane);
        __syncwarp();
        const View& v = which ? a.dv : a.dk;
        __nv_bfloat16* base =
            reinterpret_cast<__nv_bfloat16*>(v.p) + b * v.b + hk * v.h + c0 + (lane & 7) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int k = 4 * i + (lane >> 3), key = j0 + (warp & 3) * 32 + k;
          if (key < a.n_kv)
            *reinterpret_cast<uint4*>(base + key * v.n) =
                *reinterpret_cast<const uint4*>(stage + k * 128 + (((lane & 7) ^ (k & 7)) << 4));
        }
      }
    } else if (ok) {
      const long long all = (long long)a.B * a.heads_kv * a.n_kv, at = (long long)bh * a.n_kv + j;
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const View& v = which ? a.dv : a.dk;
#pragma unroll
        for (int q = 0; q < HD / 64; ++q) {
          const int c0 = x * (HD / 2) + 32 * q;
          uint32_t o[32];
          if (n > 0) {
            TMEM_LD32((which ? tV : tK) + lane_off + c0, o);
            TMEM_LD_WAIT(o);
          }
          if (n == 0 || !seen) {
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = 0u;
          }
          if (j < a.n_kv) {
            const float by = which ? 1.0f : a.scale;
            if (a.splits > 1 || a.slot_of)
              store32(a.part_kv + ((2ll * split + which) * all + at) * HD + c0, o, by);
            else
              store32(reinterpret_cast<__nv_bfloat16*>(v.p) + b * v.b + j * v.n + hk * v.h + c0, o, by);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort) atomicCAS(a.status, 0, (int)BSA_ERR_TIMEOUT);
}

// -lse in log2 units and -delta of every row of every query tile, in the
// tiles' row order: HD / 8 threads per row, 16 bytes of O and dO each, four rows
// per thread so that enough loads are in flight (one row: 49 us instead of 37 for
// 200 MB).  Rows without a token, or without keys, get -inf and so P = 0.  (CTAs from
// `row_ctas` on count keys.)
template <int HD>
__global__ void __launch_bounds__(256) cross_stats(const __grid_constant__ CrossArgs a,
                                                   const __grid_constant__ CrossTiles t, unsigned row_ctas) {
  if (blockIdx.x >= row_ctas) {
    count_keys(a, (int)(blockIdx.x - row_ctas));
    return;
  }
  constexpr int G = HD / 8, kRows = 4, kGroups = 256 / G;      // kGroups * kRows divides 128
  const long long first = (long long)blockIdx.x * kGroups * kRows;
  const long long tile = first >> 7;
  const int c = (threadIdx.x % G) * 8;
  const int bh = (int)(tile / t.tiles), i = (int)(tile - (long long)bh * t.tiles);
  const int sg = (int)fdiv((uint32_t)i, t.div_tok);
  const int b = bh / a.heads_kv, h0 = (bh - b * a.heads_kv) * a.group + sg * t.pack;
  const int n0 = (i - sg * (int)t.div_tok.d) * t.tokens;
  uint4 u[kRows], v[kRows];
  float lse[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int r = (int)(first & 127) + k * kGroups + threadIdx.x / G, rt = (int)fdiv((uint32_t)r, t.div_pack);
    const int n = n0 + rt, h = h0 + r - rt * t.pack;
    u[k] = v[k] = make_uint4(0u, 0u, 0u, 0u);
    lse[k] = -INFINITY;
    if (n < a.n_q) {
      u[k] = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.o.p) + b * a.o.b +
                                                  n * a.o.n + h * a.o.h + c));
      v[k] = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.d_o.p) + b * a.d_o.b +
                                                  n * a.d_o.n + h * a.d_o.h + c));
      lse[k] = __ldg(a.lse + ((long long)b * a.heads + h) * a.n_q + n);
    }
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int r = (int)(first & 127) + k * kGroups + threadIdx.x / G;
    const uint32_t x[4] = {u[k].x, u[k].y, u[k].z, u[k].w}, y[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sum = fmaf(__uint_as_float(x[e] << 16), __uint_as_float(y[e] << 16), sum);
      sum = fmaf(__uint_as_float(x[e] & 0xffff0000u), __uint_as_float(y[e] & 0xffff0000u), sum);
    }
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (threadIdx.x % G == 0) {
      a.stats[tile * 256 + r] = lse[k] == -INFINITY ? -INFINITY : lse[k] * -1.4426950408889634f;
      a.stats[tile * 256 + 128 + r] = -sum;
    }
  }
}

template <int HD>
cudaError_t launch_dq(const CrossArgs& a, const CrossTiles& t, const CrossMaps& m, cudaStream_t st) {
  cross_tc_dq<HD><<<t.items < t.ctas ? t.items : t.ctas, kThreads, DqLayout<HD>::kAlloc, st>>>(a, t, m);
  return cudaGetLastError();
}

template <int HD>
cudaError_t launch_dkv(const CrossArgs& a, const CrossTiles& t, const CrossMaps& m, cudaStream_t st) {
  const unsigned ctas = (unsigned)(a.B * a.heads_kv * ((a.n_kv + 127) / 128) * a.splits);
  cross_tc_dkv<HD><<<ctas, kThreads, DkvLayout<HD>::kAlloc, st>>>(a, t, m);
  return cudaGetLastError();
}

template <int HD>
cudaError_t prepare() {
  const cudaError_t e = prepare_kernel(cross_tc_dq<HD>, DqLayout<HD>::kAlloc);
  return e == cudaSuccess ? prepare_kernel(cross_tc_dkv<HD>, DkvLayout<HD>::kAlloc) : e;
}

}  // namespace

cudaError_t launch_cross_tc_dq(const CrossArgs& a, const CrossTiles& t, const CrossMaps& m, int D, cudaStream_t st) {
  return D == 128 ? launch_dq<128>(a, t, m, st) : launch_dq<64>(a, t, m, st);
}
cudaError_t launch_cross_tc_dkv(const CrossArgs& a, const CrossTiles& t, const CrossMaps& m, int D, cudaStream_t st) {
  return D == 128 ? launch_dkv<128>(a, t, m, st) : launch_dkv<64>(a, t, m, st);
}
cudaError_t prepare_cross_tc_backward(int D) { return D == 128 ? prepare<128>() : prepare<64>(); }
cudaError_t launch_cross_stats(const CrossArgs& a, const CrossTiles& t, int D, cudaStream_t st) {
  const long long rows = (long long)a.B * a.heads_kv * t.tiles * 128;
  const unsigned ctas = (unsigned)(rows * (D / 8) / (256 * 4));
  const unsigned more = a.attended ? (unsigned)a.B : 0u;
  if (D == 128) cross_stats<128><<<ctas + more, 256, 0, st>>>(a, t, ctas);
  else cross_stats<64><<<ctas + more, 256, 0, st>>>(a, t, ctas);
  return cudaGetLastError();
}

}  // namespace bsa
