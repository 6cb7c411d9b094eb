// cross_tc.cu — cross attention forward on the tensor cores (bf16).
//
// One persistent CTA per SM walks over items.  Each CTA runs two streams of
// 128-row query tiles: warps 0-3 and 4-7 are the softmax of stream 0 and 1 (a
// query row per thread), warp 8 issues the TMA loads, warp 9 the MMAs, warps 10
// and 11 clear V at masked keys.  An item
// gives each stream a query tile and a run of key tiles; either the streams
// take two query tiles of one K/V head over the same keys and share every K and
// V tile in shared memory, or (few query rows) the same query tile over the two
// halves of the keys, and the partial rows are merged afterwards.
//
// TMEM (512 columns): S of stream x at 128 x, O of stream x at 256 + 128 x; P
// (bf16) overwrites the first 64 columns of S and is the A operand of the
// product with V.  The MMA order
//   S0(0) S1(0) | PV0(0) S0(1) PV1(0) S1(1) | PV0(1) S0(2) ...
// runs on over item boundaries: while the softmax warps of a stream finish a
// tile, the tensor core works for the other one, and the next tile's S is
// formed during the epilogue.  A commit after S_x(s) covers every earlier MMA,
// so a softmax warp that sees it may rescale O_x.
#include "cross_tc.cuh"

namespace bsa {
namespace {

using Regs = RegSplit<216, 72>;
constexpr float kRescale = 8.0f;   // log2 units by which a row's maximum may lag

template <int HD>
struct Layout {
  static constexpr int kTile = 128 * HD * 2;
  static constexpr int kPanel = 128 * 128;       // 128 rows x 64 columns (one TMA box)
  static constexpr int kStages = HD == 128 ? 2 : 4;         // slots of the K ring, and of the V ring
  static constexpr int kQ = 0;
  static constexpr int kRing = 2 * kTile;
  static constexpr int kStore = kRing + 2 * kStages * kTile; // 4 KB per softmax warp
  static constexpr int kBars = kStore + 8 * 4096;
  static constexpr int kQFull = 0, kQEmpty = 2, kFull = 4, kEmpty = kFull + 2 * kStages,
                       kClean = kEmpty + 2 * kStages, kS = kClean + kStages, kP = kS + 2, kO = kP + 2,
                       kFinal = kO + 2, kNumBars = kFinal + 1;
  static constexpr int kTmemSlot = kBars + kNumBars * 8;
  static constexpr int kAbort = kTmemSlot + 4;
  static constexpr int kAlloc = kAbort + 4 + 1024;   // room to align the base to 1024
};

// f(kind, x, cursor) for every event of the CTA in issue order; kind 0 is
// S = Q K^T, 1 is O += P V.  Stops and returns false when f does.
template <class F>
__device__ __forceinline__ bool for_each_event(const CrossArgs& a, const CrossTiles& t, F&& f) {
  Cursor c[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    c[x].start(a, t, x);
    if (c[x].valid(t) && !f(0, x, c[x])) return false;
  }
  while (c[0].valid(t) || c[1].valid(t)) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (!c[x].valid(t)) continue;
      if (!f(1, x, c[x])) return false;
      c[x].advance(a, t, x);
      if (c[x].valid(t) && !f(0, x, c[x])) return false;
    }
  }
  return true;
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    cross_tc_forward(const __grid_constant__ CrossArgs a, const __grid_constant__ CrossTiles t,
                     const __grid_constant__ CrossMaps maps) {
  using L = Layout<HD>;
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
      mbar_init(bar(x), x == L::kP || x == L::kP + 1 ? 128u : x >= L::kClean && x < L::kClean + L::kStages ? 2u : 1u);
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
    Regs::small();
    if (warp == 8 && lane == 0) {
      // ------------------------------------------------------------ loads
      int pos[2] = {0, 0}, nq[2] = {0, 0};
      const uint32_t q_bytes = (uint32_t)(t.pack * t.tokens * HD * 2);
      for_each_event(a, t, [&](int kind, int x, const Cursor& c) -> bool {
        const Work& w = c.w;
        if (kind == 0 && c.s == 0) {
          if (nq[x] > 0 && !mbar_wait(bar(L::kQEmpty + x), (nq[x] - 1) & 1, abort, lim)) return false;
          mbar_arrive_expect_tx(bar(L::kQFull + x), q_bytes);
          // the padding tile of an odd pair lies past the tokens and reads zeros
          const int tok = w.real ? w.tok0 : a.n_q;
#pragma unroll
          for (int p = 0; p < HD / 64; ++p)
            tma_load_4d(sb + L::kQ + x * L::kTile + p * L::kPanel, &maps.q, 64 * p, (w.real ? w.h0 : 0) * t.step_qh,
                        tok, w.b * t.step_qb, bar(L::kQFull + x));
          ++nq[x];
        }
        if (t.shared && x == 1) return true;
        if (pos[0] + pos[1] + 1 == t.hold_load && blockIdx.x == 0) return false;   // test hook: a copy that never lands
        const int use = pos[kind] / L::kStages, slot = kind * L::kStages + pos[kind] % L::kStages;
        if (use > 0 && !mbar_wait(bar(L::kEmpty + slot), (use - 1) & 1, abort, lim)) return false;
        mbar_arrive_expect_tx(bar(L::kFull + slot), L::kTile);
        const CUtensorMap* map = kind ? &maps.v : &maps.k;
        const int hc = w.hk * (kind ? t.step_vh : t.step_kh), bc = w.b * (kind ? t.step_vb : t.step_kb);
#pragma unroll
        for (int p = 0; p < HD / 64; ++p)
          tma_load_4d(sb + L::kRing + slot * L::kTile + p * L::kPanel, map, 64 * p, hc, (w.kt + c.s) * 128, bc,
                      bar(L::kFull + slot));
        ++pos[kind];
        return true;
      });
      // No copy is left in flight, also after an abort: issued copies land.
      for (int x = 0; x < 2; ++x)
        if (nq[x] > 0) mbar_wait_drain(bar(L::kQFull + x), (nq[x] - 1) & 1, lim);
      for (int y = 0; y < 2; ++y)
        for (int p = pos[y] > L::kStages ? pos[y] - L::kStages : 0; p < pos[y]; ++p)
          mbar_wait_drain(bar(L::kFull + y * L::kStages + p % L::kStages), (p / L::kStages) & 1, lim);
    } else if (warp == 9) {
      // ------------------------------------------------------------ MMAs (the whole warp waits, one lane issues)
      int pos[2] = {0, 0}, kept[2] = {0, 0}, nq[2] = {0, 0}, np[2] = {0, 0};
      auto wait = [&](uint32_t b, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(b, parity, abort, lim)) != 0;
      };
      for_each_event(a, t, [&](int kind, int x, const Cursor& c) -> bool {
        const Work& w = c.w;
        const bool own = !(t.shared && x == 1);      // else: the slot stream 0 took
        const int slot = own ? kind * L::kStages + pos[kind] % L::kStages : kept[kind];
        const uint32_t src = sb + L::kRing + slot * L::kTile;
        if (kind == 0 && c.s == 0) {
          if (!wait(bar(L::kQFull + x), nq[x] & 1)) return false;
          ++nq[x];
        }
        if (own) {
          const int ready = kind && cleaning ? L::kClean + slot - L::kStages : L::kFull + slot;
          if (!wait(bar(ready), (pos[kind] / L::kStages) & 1)) return false;
          ++pos[kind];
          kept[kind] = slot;
        }
        if (kind == 1) {
          if (!wait(bar(L::kP + x), np[x] & 1)) return false;
          ++np[x];
        }
        tc_fence_after();
        const uint32_t tS = tmem + 128u * x, tO = tmem + 256u + 128u * x;
        if (elect_one()) {
          if (kind == 0) {
            mma_rows<HD>(tS, sb + L::kQ + x * L::kTile, src);
            tc_commit(bar(L::kS + x));
            if (c.s == w.n - 1) tc_commit(bar(L::kQEmpty + x));
          } else {
            mma_cols<HD>(tO, tS, 32u, src, c.s > 0);
            if (c.s == w.n - 1) tc_commit(bar(L::kO + x));
          }
          if (!t.shared || x == 1) tc_commit(bar(L::kEmpty + slot));
        }
        __syncwarp();
        return true;
      });
      // Every MMA issued is complete before TMEM is released, also after an abort.
      if (elect_one()) tc_commit(bar(L::kFinal));
      mbar_wait_drain(bar(L::kFinal), 0, lim);
    } else if (warp >= 10 && cleaning) {
      // ------------------------------------------------------------ cleaning of V
      // What V holds at keys that are not attended must not enter, not even
      // times 0: warps 10 and 11 write zeros over those rows (64 rows each)
      // while the tile waits for its turn.  (Rows past n_kv are zeros.)
      int pos = 0;
      for_each_event(a, t, [&](int kind, int x, const Cursor& c) -> bool {
        if (kind == 0 || (t.shared && x == 1)) return true;
        const int slot = pos % L::kStages, j0 = (c.w.kt + c.s) * 128, keys = cross_keys(a, c.w.b);
        const bool hidden = a.key_mask != nullptr || j0 + 128 > keys;
        uint4 m;
        if (hidden) m = seen_bits(a, c.w.b, j0, keys, lane);
        if (!__all_sync(0xffffffffu, mbar_wait(bar(L::kFull + L::kStages + slot), (pos / L::kStages) & 1, abort, lim)))
          return false;
        if (hidden) zero_hidden_rows<HD>(sm + L::kRing + (L::kStages + slot) * L::kTile, m, 2 * (warp - 10), lane);
        if (lane == 0) mbar_arrive(bar(L::kClean + slot));
        ++pos;
        return true;
      });
    }
  } else {
    // ------------------------------------------------------------ softmax
    Regs::rows();
    const int x = warp >> 2, r = (warp & 3) * 32 + lane;    // stream, query row of the tile (TMEM lane)
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + 128u * x + lane_off, tO = tmem + 256u + 128u * x + lane_off;
    const int rt = (int)fdiv((uint32_t)r, t.div_pack), rg = r - rt * t.pack;   // token and head of the row
    const long long rows = cross_rows(a);
    int gs = 0, gi = 0;       // steps and items done (barrier phases)
    bool ok = true;
    for (int it = blockIdx.x; it < t.items && ok; it += gridDim.x) {
      const Work w = decode(a, t, it, x);
      const int keys = cross_keys(a, w.b);
      float m_run = -INFINITY, l = 0.f;
      for (int s = 0; s < w.n; ++s, ++gs) {
        const int j0 = (w.kt + s) * 128;
        const bool partial = a.key_mask != nullptr || j0 + 128 > keys;
        uint4 mw;
        if (partial) mw = seen_bits(a, w.b, j0, keys, lane);
        if (!__all_sync(0xffffffffu, mbar_wait(bar(L::kS + x), gs & 1, abort, lim))) { ok = false; break; }
        tc_fence_after();
        uint32_t sr[128];
        TMEM_LD32(tS + 0, (sr + 0));
        TMEM_LD32(tS + 32, (sr + 32));
        TMEM_LD32(tS + 64, (sr + 64));
        TMEM_LD32(tS + 96, (sr + 96));
        TMEM_LD_WAIT((sr + 0));
        TMEM_LD_WAIT((sr + 32));
        TMEM_LD_WAIT((sr + 64));
        TMEM_LD_WAIT((sr + 96));
        if (partial) {
          const uint32_t w4[4] = {mw.x, mw.y, mw.z, mw.w};
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (!((w4[c >> 5] >> (c & 31)) & 1u)) sr[c] = __float_as_uint(-INFINITY);
        }
        float mp[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) mp[k] = __uint_as_float(sr[k]);
#pragma unroll
        for (int c = 8; c < 128; ++c) mp[c & 7] = fmaxf(mp[c & 7], __uint_as_float(sr[c]));
        const float mx = fmaxf(fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3])),
                               fmaxf(fmaxf(mp[4], mp[5]), fmaxf(mp[6], mp[7])));
        const float m_cand = mx * a.scale_log2;
        const bool need = m_cand > m_run + kRescale;
        const bool any_need = __any_sync(0xffffffffu, need);
        float scale = 1.f;
        if (any_need) {
          const float m_new = need ? m_cand : m_run;
          scale = need ? fast_ex2(m_run - m_new) : 1.f;
          l *= scale;
          m_run = m_new;
        }
        const float m_use = m_run == -INFINITY ? 0.f : m_run;
        const float2 sl2 = make_float2(a.scale_log2, a.scale_log2), neg_m = make_float2(-m_use, -m_use);
        float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        uint32_t pk[64];
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          const float2 e = fma2(make_float2(__uint_as_float(sr[2 * c]), __uint_as_float(sr[2 * c + 1])), sl2, neg_m);
          const float2 p = make_float2(fast_ex2(e.x), fast_ex2(e.y));
          acc[c & 3] = add2(acc[c & 3], p);
          pk[c] = pack_bf16x2(p.x, p.y);
        }
        const float2 a03 = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
        l += a03.x + a03.y;
        TMEM_ST32(tS + 0, (pk + 0));
        TMEM_ST32(tS + 32, (pk + 32));
        // this S was committed after the previous product with V, so O is at rest
        if (any_need && s > 0) {
#pragma unroll
          for (int c0 = 0; c0 < HD; c0 += 32) {
            uint32_t o[32];
            TMEM_LD32(tO + c0, o);
            TMEM_LD_WAIT(o);
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * scale);
            TMEM_ST32(tO + c0, o);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar(L::kP + x));
      }
      if (!ok) break;
      if (w.n > 0) {
        if (!__all_sync(0xffffffffu, mbar_wait(bar(L::kO + x), gi & 1, abort, lim))) { ok = false; break; }
        tc_fence_after();
        ++gi;
      }
      // Rows of the tile that stand for a (head, token): written; a tile
      // without keys gives zeros.
      const int n = w.tok0 + rt, h = w.h0 + rg;
      const bool row = w.real && rt < t.tokens && n < a.n_q;
      const long long at = ((long long)w.b * a.heads + h) * a.n_q + n;
      if (a.splits > 1) {
        const long long p = w.split * rows + at;
        if (w.n > 0) {
#pragma unroll
          for (int c0 = 0; c0 < HD; c0 += 32) {
            uint32_t o[32];
            TMEM_LD32(tO + c0, o);
            TMEM_LD_WAIT(o);
            if (row) {
#pragma unroll
              for (int c = 0; c < 8; ++c)
                reinterpret_cast<uint4*>(a.part_o + p * HD + c0)[c] =
                    make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
            }
          }
        }
        if (row) a.part_ml[p] = make_float2(m_run, l);
      } else {
        const float inv = m_run == -INFINITY ? 0.f : 1.f / l;
#pragma unroll
        for (int c0 = 0; c0 < HD; c0 += 64) {
          uint32_t o[64];
          if (w.n > 0) {
            TMEM_LD32(tO + c0, (o + 0));
            TMEM_LD32(tO + c0 + 32, (o + 32));
            TMEM_LD_WAIT((o + 0));
            TMEM_LD_WAIT((o + 32));
          } else {
#pragma unroll
            for (int c = 0; c < 64; ++c) o[c] = 0u;
          }
          // the warp's staging holds 64 columns: the store before has to have read it
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
          store_rows64(a, t, &maps.out, a.o, w, sm + L::kStore + warp * 4096, (warp & 3) * 32, c0, o, inv, lane);
        }
        if (row && a.lse) a.lse[at] = (m_run + __log2f(l)) * 0.69314718055994531f;
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
cudaError_t launch(const CrossArgs& a, const CrossTiles& t, const CrossMaps& m, cudaStream_t st) {
  const cudaError_t e = prepare_kernel(cross_tc_forward<HD>, Layout<HD>::kAlloc);
  if (e != cudaSuccess) return e;
  cross_tc_forward<HD><<<t.items < t.ctas ? t.items : t.ctas, kThreads, Layout<HD>::kAlloc, st>>>(a, t, m);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cross_tc_forward(const CrossArgs& a, const CrossTiles& t, const CrossMaps& m, int D,
                                    cudaStream_t st) {
  return D == 128 ? launch<128>(a, t, m, st) : launch<64>(a, t, m, st);
}

}  // namespace bsa
