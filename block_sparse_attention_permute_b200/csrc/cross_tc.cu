// cross_tc.cu — cross attention forward on the tensor cores (bf16).
//
// One persistent CTA per SM walks over items.  Each CTA runs two streams of
// 128-row query tiles: warps 0-3 and 4-7 are the softmax of stream 0 and 1 (a
// query row per thread), warp 8 issues the TMA loads, warp 9 the MMAs, warps 10
// and 11 clear V at masked keys.  An item gives each stream a query tile and a
// run of key tiles; either the streams take two query tiles of one K/V head over
// the same keys and share every K and V tile in shared memory, or (few query
// rows) the same query tile over the two halves of the keys, and the partial
// rows are merged afterwards.
//
// A step is 128 keys.  TMEM (512 columns): S of stream x at 128 x, O of stream x
// at 256 + 128 x; P (bf16) overwrites the first 64 columns of S and is the A
// operand of the product with V.  The MMA order
//   S0(0) S1(0) | PV0(0) S0(1) PV1(0) S1(1) | PV0(1) S0(2) ...
// runs on over item boundaries: while the softmax warps of a stream work on its
// S, the tensor core works for the other one.  A commit after S_x(s) covers every
// earlier MMA, so a softmax warp that sees it may rescale O_x.  (Steps of 64 keys
// with two buffers of S, which let S run ahead, were 40% slower: an MMA of N = 64
// takes nearly as long as one of N = 128 when A comes from shared memory, 75
// against 84 cycles.)
//
// Measured on B200: 32 760 queries x 512 keys x 12 heads of 128 in 125 us (822
// TFLOP/s, 0.51 of cuBLAS's burst rate) in a sustained loop, which runs at the
// 1000 W cap and 1.7 GHz, 110 us in a short burst; tensor pipe 47% busy, MUFU 48%.
// One query of 32 heads over 8 heads x 32 760 keys, batch 2: 45 to 47 us, 5.1 to 5.3 TB/s.
// Bound by a stream's chain S -> softmax (1650 cycles, 1024 of them MUFU) -> PV
// and by MMAs that read both operands from shared memory (84 cycles, not 64).  A
// part of the exponentials as a polynomial on the FMA pipe did not pay (25%: 127.7
// against 124.8 us).
#include "cross_tc.cuh"

namespace bsa {
namespace {

constexpr float kRescale = 8.0f;   // log2 units by which a row's maximum may lag
constexpr int kStep = 128;         // keys of a step

template <int HD, bool SHARED>
struct Layout {
  static constexpr int kTile = 128 * HD * 2, kPanel = 128 * 128;   // a tile, its 64-column panels (TMA boxes)
  // Streams that share K and V hold a K tile from S0 to S1 and a V tile from
  // PV0 to PV1, whose successor is wanted one S later: one K slot, two V slots and
  // the next item's Q; streams with keys of their own take more of each instead.
  static constexpr int kItems = SHARED ? 2 : 1;
  static constexpr int kSlotsK = HD == 128 ? (SHARED ? 1 : 2) : 4, kSlotsV = HD == 128 ? (SHARED ? 2 : 3) : 4;
  static constexpr int kSlots = kSlotsK + kSlotsV;
  static constexpr int kQ = 0;                                     // 2 streams x kItems
  static constexpr int kRing = 2 * kItems * kTile;                 // K slots, then V slots
  static constexpr int kBars = kRing + kSlots * kTile;
  // Q: [stream + 2 * (item % kItems)]; full, empty: [slot]; clean: [V slot]; S, P, O: [stream]
  static constexpr int kQFull = 0, kQEmpty = 4, kFull = 8, kEmpty = kFull + kSlots, kClean = kEmpty + kSlots,
                       kS = kClean + kSlotsV, kP = kS + 2, kO = kP + 2, kFinal = kO + 2, kNumBars = kFinal + 1;
  // ring slot of the p-th K (kind 0) or V tile, and how often it was used before
  static __device__ __forceinline__ int slot(int kind, int p) { return kind ? kSlotsK + p % kSlotsV : p % kSlotsK; }
  static __device__ __forceinline__ int use(int kind, int p) { return kind ? p / kSlotsV : p / kSlotsK; }
  static constexpr int kTmemSlot = kBars + kNumBars * 8;
  static constexpr int kAbort = kTmemSlot + 4;
  static constexpr int kAlloc = kAbort + 4 + 1024;   // room to align the base to 1024
};

// f(kind, x, cursor) for every event of the CTA in issue order; kind 0 is
// S = Q K^T, 1 is O += P V.  Stops and returns false when f does.  (One call
// site: the kernel has to fit the instruction cache.)
template <class F>
__device__ __forceinline__ void for_each_event(const CrossArgs& a, const CrossTiles& t, F&& f) {
  Cursor ahead, c;
  ahead.start(a, t);
  c = ahead;
  for (int k = 0; k < 1 || c.valid(t); ++k) {
#pragma unroll 1
    for (int e = k < 1 ? 1 : 0; e < 4; e += k < 1 ? 2 : 1) {
      const int x = e >> 1, kind = 1 - (e & 1);
      const Cursor& y = kind ? c : ahead;
      if (!y.valid(t) || !y.active(x)) continue;
      if (!f(kind, x, y)) return;
    }
    if (k >= 1) c.advance(a, t);
    if (ahead.valid(t)) ahead.advance(a, t);
  }
}

template <int HD, bool SHARED>
__global__ void __launch_bounds__(kThreads, 1)
    cross_tc_forward(const __grid_constant__ CrossArgs a, const __grid_constant__ CrossTiles t,
                     const __grid_constant__ CrossMaps maps) {
  using L = Layout<HD, SHARED>;
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
      mbar_init(bar(x), x >= L::kP && x < L::kP + 2                                             ? 128u
                        : x >= L::kQEmpty && x < L::kQEmpty + 4                               ? 4u
                        : x >= L::kClean && x < L::kClean + L::kSlotsV                          ? 2u
                                                                                                : 1u);
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
      int pos[2] = {0, 0}, nq[2] = {0, 0};
      const uint32_t q_bytes = (uint32_t)(t.pack * t.tokens * HD * 2);
      for_each_event(a, t, [&](int kind, int x, const Cursor& c) -> bool {
        const Work& w = c.w;
        if (kind == 0 && c.s == 0) {
          const int i = x ? nq[1]++ : nq[0]++, q = x + 2 * (i % L::kItems);
          if (i >= L::kItems && !mbar_wait(bar(L::kQEmpty + q), (i / L::kItems - 1) & 1, abort, lim)) {
            --(x ? nq[1] : nq[0]);
            return false;
          }
          mbar_arrive_expect_tx(bar(L::kQFull + q), q_bytes);
          // the padding tile of an odd pair lies past the tokens and reads zeros
          const RowTile r = row_tile(a, t, w, x);
#pragma unroll
          for (int p = 0; p < HD / 64; ++p)
            tma_load_4d(sb + L::kQ + q * L::kTile + p * L::kPanel, &maps.q, 64 * p, (r.real ? r.h0 : 0) * t.step_qh,
                        r.real ? r.tok0 : a.n_q, w.b * t.step_qb, bar(L::kQFull + q));
        }
        if (SHARED && x == 1) return true;
        if (pos[0] + pos[1] + 1 == t.hold_load && blockIdx.x == 0) return false;   // test hook: a copy that never lands
        const int p = kind ? pos[1] : pos[0];
        const int use = L::use(kind, p), slot = L::slot(kind, p);
        if (use > 0 && !mbar_wait(bar(L::kEmpty + slot), (use - 1) & 1, abort, lim)) return false;
        mbar_arrive_expect_tx(bar(L::kFull + slot), L::kTile);
        const CUtensorMap* map = kind ? &maps.v : &maps.k;
        const int hc = w.hk * (kind ? t.step_vh : t.step_kh), bc = w.b * (kind ? t.step_vb : t.step_kb);
#pragma unroll
        for (int y = 0; y < HD / 64; ++y)
          tma_load_4d(sb + L::kRing + slot * L::kTile + y * L::kPanel, map, 64 * y, hc, c.key_step(x) * kStep, bc,
                      bar(L::kFull + slot));
        if (kind) ++pos[1];
        else ++pos[0];
        return true;
      });
      // No copy is left in flight, also after an abort: issued copies land.
      for (int x = 0; x < 2; ++x) {
        for (int i = nq[x] > L::kItems ? nq[x] - L::kItems : 0; i < nq[x]; ++i)
          mbar_wait_drain(bar(L::kQFull + x + 2 * (i % L::kItems)), (i / L::kItems) & 1, lim);
        const int slots = x ? L::kSlotsV : L::kSlotsK;
        for (int p = pos[x] > slots ? pos[x] - slots : 0; p < pos[x]; ++p)
          mbar_wait_drain(bar(L::kFull + L::slot(x, p)), L::use(x, p) & 1, lim);
      }
    } else if (warp == 9) {
      // ------------------------------------------------------------ MMAs (the whole warp waits, one lane issues)
      // Its instructions between two events are on every stream's critical path,
      // so it keeps no more than counters: what an item is, only its step counts
      // say here.
      auto wait = [&](int b, int phase) {
        return __all_sync(0xffffffffu, mbar_wait(bar(b), phase & 1, abort, lim)) != 0;
      };
      int pk = 0, pv = 0, items[2] = {0, 0}, g[2] = {0, 0};   // K and V tiles taken, items and products with V per stream
      // S of stream x for the next step (c.s == s)
      auto score = [&](int x, bool first) -> bool {
        const int slot = L::slot(0, SHARED && x ? pk - 1 : pk);
        if (!(SHARED && x)) {
          if (!wait(L::kFull + slot, L::use(0, pk))) return false;
          ++pk;
        }
        if (first) {
          if (!wait(L::kQFull + x + 2 * (items[x] % L::kItems), items[x] / L::kItems)) return false;
          ++items[x];
        }
        tc_fence_after();
        if (elect_one()) {
          mma_rows<HD>(tmem + 128u * x, sb + L::kQ + (x + 2 * ((items[x] - 1) % L::kItems)) * L::kTile,
                       sb + L::kRing + slot * L::kTile);
          tc_commit(bar(L::kS + x));
          if (!SHARED || x) tc_commit(bar(L::kEmpty + slot));
        }
        __syncwarp();
        return true;
      };
      // O of stream x += P V
      auto product = [&](int x, bool first, bool last) -> bool {
        const int p = SHARED && x ? pv - 1 : pv, slot = L::slot(1, p);
        if (!(SHARED && x)) {
          // V is ready once it is cleaned
          if (!wait(cleaning ? L::kClean + slot - L::kSlotsK : L::kFull + slot, L::use(1, p))) return false;
          ++pv;
        }
        if (!wait(L::kP + x, g[x])) return false;
        ++g[x];
        tc_fence_after();
        if (elect_one()) {
          mma_cols<HD>(tmem + 256u + 128u * x, tmem + 128u * x, 32u, sb + L::kRing + slot * L::kTile, !first);
          if (last) tc_commit(bar(L::kO + x));
          if (!SHARED || x) tc_commit(bar(L::kEmpty + slot));
        }
        __syncwarp();
        return true;
      };
      Cursor c;
      c.start(a, t);
      int s = 0, n[2] = {0, 0}, m[2] = {0, 0};       // step, step counts of this item and of the next step's
      bool ok = true, some = c.valid(t);
      if (some) n[0] = c.w.steps(0), n[1] = c.w.steps(1);
      for (bool head = true; ok && some; head = false) {
        // the step after this one (the first of the next item after the last)
        bool more = true;
        int sn = s + 1;
        m[0] = n[0], m[1] = n[1];
        if (head) {
          sn = 0;
        } else if (sn == n[0]) {
          c.s = n[0] - 1;
          c.advance(a, t);
          sn = 0;
          more = c.valid(t);
          if (more) m[0] = c.w.steps(0), m[1] = c.w.steps(1);
        }
#pragma unroll
        for (int x = 0; x < 2 && ok; ++x) {
          if (!head && s < n[x]) ok = product(x, s == 0, s + 1 == n[x]);
          if (ok && more && sn < m[x]) ok = score(x, sn == 0);
        }
        s = sn, n[0] = m[0], n[1] = m[1], some = more;
      }
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
        if (kind == 0 || (SHARED && x == 1)) return true;
        const int slot = L::slot(1, pos), j0 = c.key_step(x) * kStep + 64 * (warp - 10);
        const uint32_t hidden0 = ~seen_word(a, c.w.b, j0, c.w.keys, lane), hidden1 = ~seen_word(a, c.w.b, j0 + 32, c.w.keys, lane);
        if (!__all_sync(0xffffffffu, mbar_wait(bar(L::kFull + slot), L::use(1, pos) & 1, abort, lim))) return false;
        uint8_t* rows = sm + L::kRing + slot * L::kTile + 64 * (warp - 10) * 128;
        if (hidden0) zero_rows<HD>(rows, L::kPanel, hidden0, lane);
        if (hidden1) zero_rows<HD>(rows + 32 * 128, L::kPanel, hidden1, lane);
        if (lane == 0) mbar_arrive(bar(L::kClean + slot - L::kSlotsK));
        ++pos;
        return true;
      });
    }
  } else {
    // ------------------------------------------------------------ softmax
    take_row_registers();
    const int x = warp >> 2, r = (warp & 3) * 32 + lane;    // stream, query row of the tile (TMEM lane)
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + 128u * x + lane_off, tO = tmem + 256u + 128u * x + lane_off;
    const int rt = (int)fdiv((uint32_t)r, t.div_pack), rg = r - rt * t.pack;   // token and head of the row
    const long long rows = cross_rows(a);
    const float2 sl2 = make_float2(a.scale_log2, a.scale_log2);
    int g = 0, items = 0;       // steps and items done (barrier phases)
    bool ok = true;
    auto wait = [&](int b, int phase) {
      return __all_sync(0xffffffffu, mbar_wait(bar(b), phase & 1, abort, lim)) != 0;
    };
    // The stores of an item's rows read the place of its Q, which goes back to
    // the loads once they have: looked at a step later, not waited for.
    int held = 0;               // items done whose Q buffer has not gone back
    auto release = [&]() {
      if (held == items) return;
      if (lane == 0) {
        bulk_wait_read<0>();
        mbar_arrive(bar(L::kQEmpty + x + 2 * (held % L::kItems)));
      }
      ++held;
    };
    Work next = decode(a, t, min((int)blockIdx.x, t.items - 1));
    for (int it = blockIdx.x; it < t.items && ok; it += gridDim.x) {
      const Work w = next;
      const int n = w.steps(x), k0 = w.first(x);
      float m_run = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int s = 0; s < n; ++s, ++g) {
        const int j0 = (k0 + s) * kStep;
        uint32_t seen[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
        if (a.key_mask != nullptr || j0 + kStep > w.keys) {
#pragma unroll
          for (int i = 0; i < 4; ++i) seen[i] = seen_word(a, w.b, j0 + 32 * i, w.keys, lane);
        }
        if (!wait(L::kS + x, g)) { ok = false; break; }
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
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (seen[i] == 0xffffffffu) continue;
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (!((seen[i] >> c) & 1u)) sr[32 * i + c] = __float_as_uint(-INFINITY);
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
        const float2 neg_m = make_float2(-m_use, -m_use);
        // P is rounded to bf16, the type of V, as tcgen05 multiplies 16-bit operands of one
        // type (tf32 for both would halve the rate and double V's bytes); the sum l takes
        // P unrounded.
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
        if (any_need && s > 0) {      // this S was committed after the previous product with V: O is at rest
#pragma unroll 1
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
        if (s == 0) release();
      }
      if (!ok) break;
      if (it + (int)gridDim.x < t.items) next = decode(a, t, it + gridDim.x);
      const RowTile q = row_tile(a, t, w, x);
      if (n > 0) {
        if (!wait(L::kO + x, items)) { ok = false; break; }
        tc_fence_after();
      }
      // Rows of the tile that stand for a (head, token) are written.
      const int tok = q.tok0 + rt, h = q.h0 + rg;
      const bool row = q.real && rt < t.tokens && tok < a.n_q;
      const long long at = ((long long)w.b * a.heads + h) * a.n_q + tok;
      if (a.splits > 1 || n == 0) {
        // a partial, unnormalised, or (no key) zeros
        const long long p = (long long)(SHARED ? w.split : 2 * w.split + x) * rows + at;
        if (a.splits > 1) {
          if (n > 0) {
#pragma unroll 1
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
        } else if (row) {
          uint4* d = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.o.p) + w.b * a.o.b + tok * a.o.n +
                                              h * a.o.h);
#pragma unroll 1
          for (int c = 0; c < HD / 8; ++c) d[c] = make_uint4(0u, 0u, 0u, 0u);
        }
      } else {
        // every MMA that reads the item's Q is done: its place serves the stores
        const float inv = m_run == -INFINITY ? 0.f : 1.f / l;
        uint8_t* stage = sm + L::kQ + (x + 2 * (items % L::kItems)) * L::kTile + (warp & 3) * (L::kTile / 4);
#pragma unroll 1
        for (int c0 = 0; c0 < HD; c0 += 64) {
          uint32_t o[64];
          TMEM_LD32(tO + c0, (o + 0));
          TMEM_LD32(tO + c0 + 32, (o + 32));
          TMEM_LD_WAIT((o + 0));
          TMEM_LD_WAIT((o + 32));
          stage_rows64(stage + c0 * 64, o, inv, lane);
        }
        store_rows<HD>(a, t, &maps.out, a.o, w.b, q, stage, (warp & 3) * 32, lane);
      }
      if (row && a.splits == 1 && a.lse) a.lse[at] = (m_run + __log2f(l)) * 0.69314718055994531f;
      if (n > 0) {
        release();
        ++items;
        if (L::kItems == 1) release();     // the next item's first step needs the place
      }
      tc_fence_before();
    }
    release();
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

template <int HD, bool SHARED>
cudaError_t launch(const CrossArgs& a, const CrossTiles& t, const CrossMaps& m, cudaStream_t st) {
  cross_tc_forward<HD, SHARED>
      <<<t.items < t.ctas ? t.items : t.ctas, kThreads, Layout<HD, SHARED>::kAlloc, st>>>(a, t, m);
  return cudaGetLastError();
}

template <int HD, bool SHARED>
cudaError_t prepare() {
  return prepare_kernel(cross_tc_forward<HD, SHARED>, Layout<HD, SHARED>::kAlloc);
}

}  // namespace

cudaError_t launch_cross_tc_forward(const CrossArgs& a, const CrossTiles& t, const CrossMaps& m, int D,
                                    cudaStream_t st) {
  if (t.shared) return D == 128 ? launch<128, true>(a, t, m, st) : launch<64, true>(a, t, m, st);
  return D == 128 ? launch<128, false>(a, t, m, st) : launch<64, false>(a, t, m, st);
}

cudaError_t prepare_cross_tc_forward(const CrossTiles& t, int D) {
  if (t.shared) return D == 128 ? prepare<128, true>() : prepare<64, true>();
  return D == 128 ? prepare<128, false>() : prepare<64, false>();
}

}  // namespace bsa
