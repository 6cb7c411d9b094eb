// cross.cuh — argument block and launchers of the cross attention kernels
// (internal; the public interface is include/bsa.h).
#pragma once
#include "common.cuh"
#include "views.cuh"

namespace bsa {

// One cross attention.  Rows are the (head, token) pairs of Q that share one
// head of K and V: row r of K/V head hk is head hk * group + r / n_q, token
// r % n_q.  Per-row buffers are indexed by (b * heads + head) * n_q + token,
// which for one (b, hk) is a contiguous range in the order of r.
struct CrossArgs {
  View q, k, v, o, d_o, dq, dk, dv;
  const int32_t* kv_len;     // [B] or null
  const uint8_t* key_mask;   // [B, n_kv] or null
  float* lse;                // [B, heads, n_q] (forward: out or null)
  float* delta;              // [B, heads, n_q] row sums of d_o * o (fp32 backward)
  float* stats;              // [query tiles][2][128]: -lse in log2 units (-inf: P = 0), -delta (bf16 backward)
  // Key-split partials of the forward: split s of a row holds the unnormalised
  // output, its maximum in log2 units and its sum.  (Also the partials of dQ.)
  float* part_o;             // [splits, rows, D]
  float2* part_ml;           // [splits, rows]
  // Row-split partials of dK and dV: [splits, 2, B, heads_kv, n_kv, D].
  float* part_kv;
  // With the attended keys gathered (k and v then are copies without gaps, kv_len
  // their counts, key_mask null): place of each key among them, -1 if none.  dK and
  // dV then always go through part_kv.
  int32_t* slot_of;          // [B, n_kv] or null
  int32_t* attended;         // [B] attended keys, 2 for more (backward with a key mask) or null
  int B, n_q, n_kv, heads, heads_kv, group;
  int splits;                // of the kernel at hand
  int split_len;             // key tiles or steps (forward, dQ) or row tiles (dK, dV) per split
  float scale, scale_log2;   // softmax scale, and times log2(e)
  int32_t* status;
};

__host__ __device__ __forceinline__ long long cross_rows(const CrossArgs& a) {
  return (long long)a.B * a.heads * a.n_q;
}

// Keys of batch element b that can be attended: kv_len[b], clamped to [0, n_kv]
// (and recorded, status BSA_ERR_BAD_INDEX, where that changes it).
__device__ __forceinline__ int cross_keys(const CrossArgs& a, int b) {
  if (a.kv_len == nullptr) return a.n_kv;
  const int n = __ldg(a.kv_len + b), c = min(max(n, 0), a.n_kv);
  if (c != n) atomicCAS(a.status, 0, (int)BSA_ERR_BAD_INDEX);
  return c;
}

// Whether batch element b attends exactly one key.  Its P is 1 and its dS 0, exactly,
// which P from a rounded lse and delta from a rounded O would miss by an ulp.
__device__ __forceinline__ bool one_key(const CrossArgs& a, int b, int keys) {
  return (a.attended ? __ldg(a.attended + b) : keys) == 1;
}

// attended[b] under the key mask, by a CTA of 256 threads: 4096 keys a time, until
// there are two.
__device__ __forceinline__ void count_keys(const CrossArgs& a, int b) {
  const int keys = cross_keys(a, b);
  const uint8_t* mask = a.key_mask + (long long)b * a.n_kv;
  int n = 0;
  for (int j0 = 0; j0 < keys && n < 2; j0 += 4096) {
    int mine = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int j = j0 + 256 * i + (int)threadIdx.x;
      mine += j < keys && __ldg(mask + j) != 0;
    }
    n += __syncthreads_count(mine > 0) + __syncthreads_count(mine > 1);
  }
  if (threadIdx.x == 0) a.attended[b] = min(n, 2);
}

// Schedule of the tensor-core kernels.  A query tile is 128 rows: `tokens`
// tokens of `pack` heads that share a K/V head (few tokens: more heads, so that
// fewer rows are empty), heads fastest.
struct CrossTiles {
  int tiles;        // query tiles of one (batch element, K/V head)
  int tokens, pack; // tokens * pack <= 128
  int bulk_out;     // a warp's 32 rows are whole tokens: the output goes by TMA (map `out`, 32 rows a box)
  int shared;       // streams take two query tiles over the same keys (else one over two key runs)
  int step;         // keys of a step (CrossArgs::split_len counts these)
  int items;        // (batch element, K/V head, split, item of it), the last fastest
  int ctas;         // CTAs at a time (one per SM)
  FastDiv div_items, div_splits, div_hkv, div_tok, div_pack;
  int step_qb, step_qh, step_kb, step_kh, step_vb, step_vh, step_ob, step_oh;   // 0 along an axis the view repeats, else 1
  long long wait_limit;   // bound of every in-kernel wait, SM cycles (0 = default)
  int hold_load;          // test hook: n > 0 = CTA 0 never issues its n-th K/V copy
};
// Tensor maps (d, head, token, batch) of the views.
struct CrossMaps {
  CUtensorMap q, k, v, d_o, out;   // out: o of the forward, dq of the backward
};

// The prepare functions run once per device before a kernel's first launch.
// cross_tc.cu (bf16)
cudaError_t prepare_cross_tc_forward(const CrossTiles& t, int D);
cudaError_t launch_cross_tc_forward(const CrossArgs& a, const CrossTiles& t, const CrossMaps& m, int D,
                                    cudaStream_t st);
// cross_tc_bwd.cu (bf16; tiles with pack * tokens == 128)
cudaError_t prepare_cross_tc_backward(int D);
cudaError_t launch_cross_tc_dq(const CrossArgs& a, const CrossTiles& t, const CrossMaps& m, int D, cudaStream_t st);
cudaError_t launch_cross_tc_dkv(const CrossArgs& a, const CrossTiles& t, const CrossMaps& m, int D, cudaStream_t st);
cudaError_t launch_cross_stats(const CrossArgs& a, const CrossTiles& t, int D, cudaStream_t st);
// cross_f32.cu (fp32)
constexpr int kCrossF32Rows = 64, kCrossF32Keys = 32;       // tile of the forward and dQ
constexpr int kCrossF32KvRows = 32, kCrossF32KvKeys = 64;   // tile of dK and dV
cudaError_t prepare_cross_f32(int D);
cudaError_t launch_cross_f32_forward(const CrossArgs& a, int D, cudaStream_t st);
cudaError_t launch_cross_f32_dq(const CrossArgs& a, int D, cudaStream_t st);
cudaError_t launch_cross_f32_dkv(const CrossArgs& a, int D, cudaStream_t st);
// cross_aux.cu
// slot_of and counts [B] from kv_len and key_mask, then the copies of K and V.
cudaError_t launch_cross_gather(const CrossArgs& a, int32_t* counts, void* k, void* v, int D, bool is_bf16,
                                cudaStream_t st);
cudaError_t launch_cross_merge(const CrossArgs& a, int D, bool is_bf16, cudaStream_t st);
cudaError_t launch_cross_delta(const CrossArgs& a, int D, cudaStream_t st);   // fp32
cudaError_t launch_cross_sum_q(const CrossArgs& a, int D, bool is_bf16, cudaStream_t st);
cudaError_t launch_cross_reduce_kv(const CrossArgs& a, int D, bool is_bf16, cudaStream_t st);

}  // namespace bsa
