// cross_aux.cu — the memory-bound passes around the cross attention kernels:
// the merge of key splits, the row sums of d_o * o, the sum of row splits.
#include "cross.cuh"

namespace bsa {
namespace {


__device__ __forceinline__ float4 in4(const float* p) {
  return __ldg(reinterpret_cast<const float4*>(p));
}
__device__ __forceinline__ void out4(float* d, float4 x) { *reinterpret_cast<float4*>(d) = x; }
__device__ __forceinline__ void out4(__nv_bfloat16* d, float4 x) {
  *reinterpret_cast<uint2*>(d) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
}

// (b, head, token) of row `at` of a per-row buffer.
__device__ __forceinline__ void row_of(const CrossArgs& a, long long at, int& b, int& h, int& n) {
  const long long bh = at / a.n_q;
  n = (int)(at - bh * a.n_q);
  b = (int)(bh / a.heads);
  h = (int)(bh - (long long)b * a.heads);
}

// One CTA per batch element: the attended keys numbered in order.
__global__ void __launch_bounds__(1024) cross_number_keys(CrossArgs a, int32_t* counts) {
  __shared__ int s_warp[32];
  const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int keys = cross_keys(a, b);
  const long long row = (long long)b * a.n_kv;
  int before = 0;
  for (int j0 = 0; j0 < a.n_kv; j0 += 1024) {
    const int j = j0 + threadIdx.x;
    const bool in = j < keys && __ldg(a.key_mask + row + j) != 0;
    const uint32_t bits = __ballot_sync(0xffffffffu, in);
    if (lane == 0) s_warp[warp] = __popc(bits);
    __syncthreads();
    int lower = 0, all = 0;
    for (int w = 0; w < 32; ++w) {
      lower += w < warp ? s_warp[w] : 0;
      all += s_warp[w];
    }
    if (j < a.n_kv) a.slot_of[row + j] = in ? before + lower + __popc(bits & ((1u << lane) - 1u)) : -1;
    before += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) counts[b] = before;
}

// Copies the attended keys' rows of K (blockIdx.y 0) and V (1) to [B, n_kv,
// heads_kv, D] without gaps (131 040 queries x 769 keys, 80% attended: 620 us with
// the two launches, 880 us when masked keys take part and are hidden), 16 bytes a thread; what lies behind a batch element's
// count stays as it is.
template <typename T, int D>
__global__ void __launch_bounds__(256) cross_gather(CrossArgs a, T* k, T* v) {
  constexpr int kPer = D * (int)sizeof(T) / 16, kEach = 16 / (int)sizeof(T);
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x, row = id / kPer;
  if (row >= (long long)a.B * a.n_kv * a.heads_kv) return;
  const int c = (int)(id % kPer) * kEach, hk = (int)(row % a.heads_kv);
  const long long bj = row / a.heads_kv;
  const int b = (int)(bj / a.n_kv), j = (int)(bj - (long long)b * a.n_kv), s = __ldg(a.slot_of + bj);
  if (s < 0) return;
  const View& from = blockIdx.y ? a.v : a.k;
  T* to = (blockIdx.y ? v : k) + (((long long)b * a.n_kv + s) * a.heads_kv + hk) * D + c;
  *reinterpret_cast<uint4*>(to) =
      __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(from.p) + b * from.b + j * from.n + hk * from.h + c));
}

// One warp per row.  With partials (O_s, m_s, l_s) of the key splits:
// M = max m_s, w_s = 2^(m_s - M), O = sum w_s O_s / sum w_s l_s, and
// lse = ln 2 (M + log2 sum w_s l_s).  A split without attended keys is told by
// l_s = 0, never by m_s = -inf: logits that are all NaN leave that maximum too, and
// their l_s = NaN has to reach the result.  A lane forms the weight of one split of 32,
// then takes its columns (D = 64: half a warp every other split) of them all.  Few
// rows leave latency as the bound, so sixteen partial rows are in flight, asked for
// before their weights are known: 5 us for 64 rows of 18 splits, 48 us with one row
// in flight.  Every sum has a fixed order.
template <typename T, int D>
__global__ void __launch_bounds__(128) cross_merge(CrossArgs a) {
  constexpr int kHalves = 128 / D, kFlight = 16;
  const long long rows = cross_rows(a), at = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (at >= rows) return;
  const int lane = threadIdx.x & 31, c = (lane % (D / 4)) * 4, first = lane / (D / 4);
  float M = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s32 = 0; s32 < a.splits; s32 += 32) {
    const int mine = s32 + lane;
    const float2 ml = mine < a.splits ? __ldg(a.part_ml + mine * rows + at) : make_float2(-INFINITY, 0.f);
    const uint32_t some = __ballot_sync(0xffffffffu, ml.y != 0.f);     // splits with attended keys
    float top = 0.f, w = 0.f;
    for (int s0 = s32; s0 < min(s32 + 32, a.splits); s0 += kFlight * kHalves) {
      float4 x[kFlight];
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int s = s0 + u * kHalves + first;
        x[u] = s < a.splits ? in4(a.part_o + (s * rows + at) * D + c) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      if (s0 == s32) {
        top = ml.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = fmaxf(top, M);
        const float base = top == -INFINITY ? 0.f : top, keep = exp2f(M - base);
        w = exp2f(ml.x - base);
        float sum = ml.y == 0.f ? 0.f : w * ml.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l = fmaf(l, keep, sum);
        acc = make_float4(acc.x * keep, acc.y * keep, acc.z * keep, acc.w * keep);
        M = top;
      }
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int s = s0 + u * kHalves + first;
        const float ws = __shfl_sync(0xffffffffu, w, s & 31);
        if ((some >> (s & 31)) & 1u)        // (a split without keys need not have written its O)
          acc = make_float4(fmaf(ws, x[u].x, acc.x), fmaf(ws, x[u].y, acc.y), fmaf(ws, x[u].z, acc.z),
                            fmaf(ws, x[u].w, acc.w));
      }
    }
  }
  if (kHalves == 2) {
    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, 16);
    acc.y += __shfl_xor_sync(0xffffffffu, acc.y, 16);
    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, 16);
    acc.w += __shfl_xor_sync(0xffffffffu, acc.w, 16);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  int b, h, n;
  row_of(a, at, b, h, n);
  if (first == 0)
    out4(reinterpret_cast<T*>(a.o.p) + b * a.o.b + n * a.o.n + h * a.o.h + c,
         make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
  if (lane == 0 && a.lse) a.lse[at] = (M + log2f(l)) * 0.69314718055994531f;
}

// A group of D / 4 threads per (token, head) row; neighbouring groups take
// neighbouring heads of a token.  (CTAs from `row_ctas` on count keys.)
template <int D>
__global__ void __launch_bounds__(256) cross_delta(CrossArgs a, unsigned row_ctas) {
  constexpr int G = D / 4;
  if (blockIdx.x >= row_ctas) {
    count_keys(a, (int)(blockIdx.x - row_ctas));
    return;
  }
  const long long rows = cross_rows(a), id = (long long)blockIdx.x * (256 / G) + threadIdx.x / G;
  float sum = 0.f;
  int b = 0, h = 0, n = 0;
  if (id < rows) {
    const long long bn = id / a.heads;
    h = (int)(id - bn * a.heads);
    b = (int)(bn / a.n_q);
    n = (int)(bn - (long long)b * a.n_q);
    const int c = (threadIdx.x % G) * 4;
    const float4 x = in4(reinterpret_cast<const float*>(a.o.p) + b * a.o.b + n * a.o.n + h * a.o.h + c);
    const float4 y = in4(reinterpret_cast<const float*>(a.d_o.p) + b * a.d_o.b + n * a.d_o.n + h * a.d_o.h + c);
    sum = x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
  }
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (id < rows && threadIdx.x % G == 0) a.delta[((long long)b * a.heads + h) * a.n_q + n] = sum;
}

// dQ from the partials of the key splits, added in order.
template <typename T, int D>
__global__ void __launch_bounds__(256) cross_sum_q(CrossArgs a) {
  constexpr int G = D / 4;
  const long long rows = cross_rows(a), at = (long long)blockIdx.x * (256 / G) + threadIdx.x / G;
  if (at >= rows) return;
  const int c = (threadIdx.x % G) * 4;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < a.splits; ++s) {
    const float4 x = in4(a.part_o + (s * rows + at) * D + c);
    acc = make_float4(acc.x + x.x, acc.y + x.y, acc.z + x.z, acc.w + x.w);
  }
  int b, h, n;
  row_of(a, at, b, h, n);
  out4(reinterpret_cast<T*>(a.dq.p) + b * a.dq.b + n * a.dq.n + h * a.dq.h + c, acc);
}

// dK and dV from the partials of the row splits, added in order (of gathered keys:
// from their places; the others get zeros).  6 splits of 12 x 512 keys x 128: 11 us.
template <typename T, int D>
__global__ void __launch_bounds__(256) cross_reduce_kv(CrossArgs a) {
  const long long all = (long long)a.B * a.heads_kv * a.n_kv;
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x, at = id / (D / 4);
  if (at >= all) return;
  const int c = (int)(id % (D / 4)) * 4, which = blockIdx.y;
  const long long bh = at / a.n_kv;
  const int j = (int)(at - bh * a.n_kv), b = (int)(bh / a.heads_kv), hk = (int)(bh % a.heads_kv);
  const int place = a.slot_of ? __ldg(a.slot_of + (long long)b * a.n_kv + j) : j;
  const long long from = bh * a.n_kv + place;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < (place < 0 ? 0 : a.splits); ++s) {
    const float4 x = in4(a.part_kv + ((2ll * s + which) * all + from) * D + c);
    acc = make_float4(acc.x + x.x, acc.y + x.y, acc.z + x.z, acc.w + x.w);
  }
  const View& v = which ? a.dv : a.dk;
  out4(reinterpret_cast<T*>(v.p) + b * v.b + j * v.n + hk * v.h + c, acc);
}

template <typename T, int D>
cudaError_t run_aux(int which, const CrossArgs& a, cudaStream_t st) {
  const long long rows = cross_rows(a), keys = (long long)a.B * a.heads_kv * a.n_kv;
  const unsigned row_ctas = (unsigned)((rows + 1024 / D - 1) / (1024 / D));
  if (which == 0) cross_merge<T, D><<<(unsigned)((rows + 3) / 4), 128, 0, st>>>(a);
  else if (which == 1) cross_sum_q<T, D><<<row_ctas, 256, 0, st>>>(a);
  else cross_reduce_kv<T, D><<<dim3((unsigned)((keys * (D / 4) + 255) / 256), 2), 256, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t run_aux(int which, const CrossArgs& a, int D, bool is_bf16, cudaStream_t st) {
  if (is_bf16) return D == 128 ? run_aux<__nv_bfloat16, 128>(which, a, st) : run_aux<__nv_bfloat16, 64>(which, a, st);
  return D == 128 ? run_aux<float, 128>(which, a, st) : run_aux<float, 64>(which, a, st);
}

}  // namespace

cudaError_t launch_cross_gather(const CrossArgs& a, int32_t* counts, void* k, void* v, int D, bool is_bf16,
                                cudaStream_t st) {
  cross_number_keys<<<a.B, 1024, 0, st>>>(a, counts);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const long long parts = (long long)a.B * a.n_kv * a.heads_kv * (D * (is_bf16 ? 2 : 4) / 16);
  const dim3 grid((unsigned)((parts + 255) / 256), 2);
  if (is_bf16) {
    __nv_bfloat16 *k2 = static_cast<__nv_bfloat16*>(k), *v2 = static_cast<__nv_bfloat16*>(v);
    if (D == 128) cross_gather<__nv_bfloat16, 128><<<grid, 256, 0, st>>>(a, k2, v2);
    else cross_gather<__nv_bfloat16, 64><<<grid, 256, 0, st>>>(a, k2, v2);
  } else {
    if (D == 128) cross_gather<float, 128><<<grid, 256, 0, st>>>(a, static_cast<float*>(k), static_cast<float*>(v));
    else cross_gather<float, 64><<<grid, 256, 0, st>>>(a, static_cast<float*>(k), static_cast<float*>(v));
  }
  return cudaGetLastError();
}
cudaError_t launch_cross_merge(const CrossArgs& a, int D, bool is_bf16, cudaStream_t st) {
  return run_aux(0, a, D, is_bf16, st);
}
cudaError_t launch_cross_sum_q(const CrossArgs& a, int D, bool is_bf16, cudaStream_t st) {
  return run_aux(1, a, D, is_bf16, st);
}
cudaError_t launch_cross_reduce_kv(const CrossArgs& a, int D, bool is_bf16, cudaStream_t st) {
  return run_aux(2, a, D, is_bf16, st);
}
cudaError_t launch_cross_delta(const CrossArgs& a, int D, cudaStream_t st) {
  const unsigned ctas = (unsigned)((cross_rows(a) + 1024 / D - 1) / (1024 / D));
  const unsigned more = a.attended ? (unsigned)a.B : 0u;
  if (D == 128) cross_delta<128><<<ctas + more, 256, 0, st>>>(a, ctas);
  else cross_delta<64><<<ctas + more, 256, 0, st>>>(a, ctas);
  return cudaGetLastError();
}

}  // namespace bsa
