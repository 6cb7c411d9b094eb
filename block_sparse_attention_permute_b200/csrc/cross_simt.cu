// cross_simt.cu — cross attention in fp32 arithmetic (forward, dQ, dK and dV).
//
// With S = scale Q K^T over the attended keys and L = log sum exp S per row:
//   O  = softmax(S) V
//   P  = exp(S - L),  dP = dO V^T,  D = rowsum(dO * O),  dS = P * (dP - D)
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO.
// 128 threads form a tile of logits, 64 query rows by 32 keys (dK and dV: 64 keys
// by 32 rows);
// operands lie in shared memory as rows padded by 4 floats, so that the 16-byte
// reads of eight consecutive rows fall into different banks, and come in by
// cp.async.  Bound by the FMA pipe (packed fp32 pairs) and the shared-memory reads
// that feed it; two or three small CTAs per SM cover one another's loads and
// barriers (tiles of 64 x 64 by one or two CTAs of 256 threads: 0.52 ms for a
// training step of 1560 rows x 226 keys x 12 heads of 128).
#include "cross.cuh"

namespace bsa {
namespace {

constexpr int kThreads = 128, kTx = 8;   // 16 x 8
constexpr int kKeys = kCrossSimtKeys;
constexpr int kPad = 36;         // row stride of a tile of probabilities (32 columns)

template <int D> constexpr int row_floats() { return D + 4; }
// Floats of a 32-key tile whose place a 64 x 32 tile of probabilities takes later.
template <int D> constexpr int key_floats() {
  return kKeys * row_floats<D>() > 64 * kPad ? kKeys * row_floats<D>() : 64 * kPad;
}

// Where row r (of one K/V head's rows) of a per-token tensor starts.
__device__ __forceinline__ float* row_ptr(const CrossArgs& a, const View& v, int b, int hk, long long r) {
  const int g = (int)(r / a.n_q);
  const long long n = r - (long long)g * a.n_q;
  return reinterpret_cast<float*>(v.p) + b * v.b + n * v.n + (long long)(hk * a.group + g) * v.h;
}

__device__ __forceinline__ void out4(float* d, float4 x) { *reinterpret_cast<float4*>(d) = x; }

// Starts the copy of rows r0 .. r0 + R - 1 (zeros from `end` on) of a row tensor.
template <int D, int R>
__device__ __forceinline__ void load_rows(float* s, const CrossArgs& a, const View& v, int b, int hk, long long r0,
                                          long long end) {
  constexpr int kPer = D / 4;
#pragma unroll 4
  for (int i = threadIdx.x; i < R * kPer; i += kThreads) {
    const int r = i / kPer, c = (i % kPer) * 4;
    const bool in = r0 + r < end;
    cp_async16(smem_addr(s + r * row_floats<D>() + c), row_ptr(a, v, b, hk, in ? r0 + r : 0) + c, in ? 16u : 0u);
  }
  cp_async_commit();
}

// Starts the copy of keys j0 .. j0 + 31 of K or V; keys that are not attended (bit
// of `seen` clear) read as zeros whatever they hold.  (The caller commits.)
template <int D>
__device__ __forceinline__ void load_keys(float* s, const View& v, int b, int hk, int j0, uint32_t seen) {
  constexpr int kPer = D / 4;
  const float* base = reinterpret_cast<const float*>(v.p) + b * v.b + hk * v.h;
#pragma unroll 4
  for (int i = threadIdx.x; i < kKeys * kPer; i += kThreads) {
    const int r = i / kPer, c = (i % kPer) * 4;
    const bool in = (seen >> r) & 1u;
    cp_async16(smem_addr(s + r * row_floats<D>() + c), base + (in ? (long long)(j0 + r) * v.n : 0) + c, in ? 16u : 0u);
  }
}

// Bit c: key j0 + c is attended.
__device__ __forceinline__ uint32_t seen_bits(const CrossArgs& a, int b, int j0, int keys) {
  const int j = j0 + (threadIdx.x & 31);
  const bool s = j < keys && (a.key_mask == nullptr || __ldg(a.key_mask + (long long)b * a.n_kv + j) != 0);
  return __ballot_sync(0xffffffffu, s);
}

// acc[i][j] = A row (ty * MR + i) . B row (tx + 8 j)
template <int D, int MR>
__device__ __forceinline__ void dot_tile(const float* A, const float* B, int ty, int tx, float (&acc)[MR][4]) {
  float2 s[MR][4];
#pragma unroll
  for (int i = 0; i < MR; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int d = 0; d < D; d += 4) {
    float4 x[MR], y[4];
#pragma unroll
    for (int i = 0; i < MR; ++i) x[i] = *reinterpret_cast<const float4*>(A + (ty * MR + i) * row_floats<D>() + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(B + (tx + 8 * j) * row_floats<D>() + d);
#pragma unroll
    for (int i = 0; i < MR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = fma2(make_float2(x[i].x, x[i].y), make_float2(y[j].x, y[j].y), s[i][j]);
        s[i][j] = fma2(make_float2(x[i].z, x[i].w), make_float2(y[j].z, y[j].w), s[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < MR; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = s[i][j].x + s[i][j].y;
}

// acc[i][q] += sum over the 32 columns k of P: P[ty * MR + i][k] B[k][tx * 4 + 32 q ..]
template <int D, int MR>
__device__ __forceinline__ void sum_tile(const float* P, const float* B, int ty, int tx, float2 (&acc)[MR][D / 16]) {
#pragma unroll 2
  for (int k = 0; k < 32; k += 4) {
    float4 p[MR];
#pragma unroll
    for (int i = 0; i < MR; ++i) p[i] = *reinterpret_cast<const float4*>(P + (ty * MR + i) * kPad + k);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        const float4 x = *reinterpret_cast<const float4*>(B + (k + kk) * row_floats<D>() + tx * 4 + 32 * q);
#pragma unroll
        for (int i = 0; i < MR; ++i) {
          const float w = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
          acc[i][2 * q] = fma2(make_float2(w, w), make_float2(x.x, x.y), acc[i][2 * q]);
          acc[i][2 * q + 1] = fma2(make_float2(w, w), make_float2(x.z, x.w), acc[i][2 * q + 1]);
        }
      }
    }
  }
}

// Over the eight threads of a row.
__device__ __forceinline__ float max8(float x) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float sum8(float x) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <int N, int M>
__device__ __forceinline__ void clear(float2 (&acc)[N][M]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int q = 0; q < M; ++q) acc[i][q] = make_float2(0.f, 0.f);
}

template <int D>
__device__ __forceinline__ void put_row(float* d, const float2 (&acc)[D / 16], int tx, float by) {
#pragma unroll
  for (int q = 0; q < D / 32; ++q)
    out4(d + tx * 4 + 32 * q,
         make_float4(acc[2 * q].x * by, acc[2 * q].y * by, acc[2 * q + 1].x * by, acc[2 * q + 1].y * by));
}

// Online softmax over the key tiles of one split; the probabilities replace K
// in shared memory for the product with V.
template <int D>
__global__ void __launch_bounds__(kThreads, 3) cross_simt_forward(CrossArgs a) {
  constexpr int R = kCrossSimtRows;
  extern __shared__ float4 smem4[];
  float* sQ = reinterpret_cast<float*>(smem4);
  float* sK = sQ + R * row_floats<D>();
  float* sV = sK + key_floats<D>();
  const int tx = threadIdx.x % kTx, ty = threadIdx.x / kTx;
  const long long rows = (long long)a.group * a.n_q;
  const int per = (int)((rows + R - 1) / R), bh = blockIdx.x / per;
  const int b = bh / a.heads_kv, hk = bh % a.heads_kv;
  const long long r0 = (long long)(blockIdx.x % per) * R;
  const int keys = cross_keys(a, b), tiles = (keys + kKeys - 1) / kKeys;
  const int t0 = blockIdx.y * a.split_len, t1 = min(tiles, t0 + a.split_len);
  load_rows<D, R>(sQ, a, a.q, b, hk, r0, rows);
  float m[4], l[4];
  float2 acc[4][D / 16];
  clear(acc);
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = -INFINITY, l[i] = 0.f;
  for (int t = t0; t < t1; ++t) {
    const uint32_t seen = seen_bits(a, b, t * kKeys, keys);
    __syncthreads();
    load_keys<D>(sK, a.k, b, hk, t * kKeys, seen);
    cp_async_commit();
    load_keys<D>(sV, a.v, b, hk, t * kKeys, seen);
    cp_async_commit();
    cp_async_wait<1>();
    __syncthreads();
    float s[4][4];
    dot_tile<D, 4>(sQ, sK, ty, tx, s);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = (seen >> (tx + 8 * j)) & 1u ? s[i][j] * a.scale_log2 : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
      const float mn = fmaxf(m[i], max8(mx));
      const float base = mn == -INFINITY ? 0.f : mn;
      const float keep = exp2f(m[i] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = exp2f(s[i][j] - base);
        sum += p;
        sK[(ty * 4 + i) * kPad + tx + 8 * j] = p;
      }
      l[i] = l[i] * keep + sum8(sum);
      m[i] = mn;
#pragma unroll
      for (int q = 0; q < D / 16; ++q) acc[i][q] = make_float2(acc[i][q].x * keep, acc[i][q].y * keep);
    }
    cp_async_wait<0>();
    __syncthreads();      // V has arrived
    sum_tile<D, 4>(sK, sV, ty, tx, acc);
  }
  cp_async_wait<0>();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long r = r0 + ty * 4 + i;
    if (r >= rows) continue;
    const long long at = ((long long)b * a.heads + (long long)hk * a.group) * a.n_q + r;
    if (a.splits > 1) {
      const long long p = blockIdx.y * cross_rows(a) + at;
      put_row<D>(a.part_o + p * D, acc[i], tx, 1.0f);
      if (tx == 0) a.part_ml[p] = make_float2(m[i], l[i]);
    } else {
      put_row<D>(row_ptr(a, a.o, b, hk, r), acc[i], tx, m[i] == -INFINITY ? 0.f : 1.f / l[i]);
      if (tx == 0 && a.lse) a.lse[at] = (m[i] + log2f(l[i])) * 0.69314718055994531f;
    }
  }
}

// P and dS of one tile: s holds Q.K on entry and P on return, dp holds dO.V on
// entry and dS / scale on return.  lse2 is in log2 units, +inf where P is 0.
__device__ __forceinline__ void grad_of(float& s, float& dp, bool seen, float lse2, float delta, float scale_log2) {
  s = seen ? exp2f(fmaf(s, scale_log2, -lse2)) : 0.f;
  dp = seen ? s * (dp - delta) : 0.f;
}

__device__ __forceinline__ float lse2_of(const CrossArgs& a, long long at, bool in) {
  const float x = in ? __ldg(a.lse + at) : -INFINITY;
  return x == -INFINITY ? INFINITY : x * 1.4426950408889634f;
}

// dQ of 64 rows, over the key tiles of one split.  dS replaces V in shared memory.
template <int D>
__global__ void __launch_bounds__(kThreads, 2) cross_simt_dq(CrossArgs a) {
  constexpr int R = kCrossSimtRows;
  extern __shared__ float4 smem4[];
  float* sQ = reinterpret_cast<float*>(smem4);
  float* sO = sQ + R * row_floats<D>();
  float* sK = sO + R * row_floats<D>();
  float* sV = sK + key_floats<D>();
  const int tx = threadIdx.x % kTx, ty = threadIdx.x / kTx;
  const long long rows = (long long)a.group * a.n_q;
  const int per = (int)((rows + R - 1) / R), bh = blockIdx.x / per;
  const int b = bh / a.heads_kv, hk = bh % a.heads_kv;
  const long long r0 = (long long)(blockIdx.x % per) * R;
  const long long at0 = ((long long)b * a.heads + (long long)hk * a.group) * a.n_q;
  const int keys = cross_keys(a, b), tiles = (keys + kKeys - 1) / kKeys;
  load_rows<D, R>(sQ, a, a.q, b, hk, r0, rows);
  load_rows<D, R>(sO, a, a.d_o, b, hk, r0, rows);
  float lse2[4], delta[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long r = r0 + ty * 4 + i;
    lse2[i] = lse2_of(a, at0 + r, r < rows);
    delta[i] = r < rows ? __ldg(a.delta + at0 + r) : 0.f;
  }
  float2 acc[4][D / 16];
  clear(acc);
  const int t0 = blockIdx.y * a.split_len, t1 = min(tiles, t0 + a.split_len);
  for (int t = t0; t < t1; ++t) {
    const uint32_t seen = seen_bits(a, b, t * kKeys, keys);
    __syncthreads();
    load_keys<D>(sK, a.k, b, hk, t * kKeys, seen);
    cp_async_commit();
    load_keys<D>(sV, a.v, b, hk, t * kKeys, seen);
    cp_async_commit();
    cp_async_wait<1>();
    __syncthreads();
    float s[4][4], dp[4][4];
    dot_tile<D, 4>(sQ, sK, ty, tx, s);
    cp_async_wait<0>();
    __syncthreads();
    dot_tile<D, 4>(sO, sV, ty, tx, dp);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        grad_of(s[i][j], dp[i][j], (seen >> (tx + 8 * j)) & 1u, lse2[i], delta[i], a.scale_log2);
        sV[(ty * 4 + i) * kPad + tx + 8 * j] = dp[i][j];
      }
    __syncwarp();         // a row of dS is written and read by the same warp
    sum_tile<D, 4>(sV, sK, ty, tx, acc);
  }
  cp_async_wait<0>();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long r = r0 + ty * 4 + i;
    if (r >= rows) continue;
    put_row<D>(a.splits > 1 ? a.part_o + (blockIdx.y * cross_rows(a) + at0 + r) * D : row_ptr(a, a.dq, b, hk, r),
               acc[i], tx, a.scale);
  }
}

// dK and dV of 64 keys, over the tiles of 32 rows of one split.
template <int D>
__global__ void __launch_bounds__(kThreads, 2) cross_simt_dkv(CrossArgs a) {
  constexpr int R = kCrossSimtKvRows, kN = kCrossSimtKvKeys;
  extern __shared__ float4 smem4[];
  float* sK = reinterpret_cast<float*>(smem4);
  float* sV = sK + kN * row_floats<D>();
  float* sQ = sV + kN * row_floats<D>();
  float* sO = sQ + R * row_floats<D>();
  float* sP = sO + R * row_floats<D>();      // P, then dS
  __shared__ float s_lse2[R], s_delta[R];
  const int tx = threadIdx.x % kTx, ty = threadIdx.x / kTx;
  const int per = (a.n_kv + kN - 1) / kN, bh = blockIdx.x / per;
  const int b = bh / a.heads_kv, hk = bh % a.heads_kv;
  const int j0 = (int)(blockIdx.x % per) * kN;
  const long long rows = (long long)a.group * a.n_q;
  const long long at0 = ((long long)b * a.heads + (long long)hk * a.group) * a.n_q;
  const int keys = cross_keys(a, b);
  const long long t0 = (long long)blockIdx.y * a.split_len;
  long long t1 = min((rows + R - 1) / R, t0 + a.split_len);
  if (j0 >= keys) t1 = t0;      // no key of this tile is attended
  const uint32_t seen0 = seen_bits(a, b, j0, keys), seen1 = seen_bits(a, b, j0 + 32, keys);
  load_keys<D>(sK, a.k, b, hk, j0, seen0);
  load_keys<D>(sK + 32 * row_floats<D>(), a.k, b, hk, j0 + 32, seen1);
  load_keys<D>(sV, a.v, b, hk, j0, seen0);
  load_keys<D>(sV + 32 * row_floats<D>(), a.v, b, hk, j0 + 32, seen1);
  cp_async_commit();
  const uint32_t mine = ((ty >= 8 ? seen1 : seen0) >> ((ty & 7) * 4)) & 15u;   // the thread's four keys
  float2 dk[4][D / 16], dv[4][D / 16];
  clear(dk);
  clear(dv);
  for (long long t = t0; t < t1; ++t) {
    __syncthreads();
    load_rows<D, R>(sQ, a, a.q, b, hk, t * R, rows);
    load_rows<D, R>(sO, a, a.d_o, b, hk, t * R, rows);
    if (threadIdx.x < R) {
      const long long r = t * R + threadIdx.x;
      s_lse2[threadIdx.x] = lse2_of(a, at0 + r, r < rows);
      s_delta[threadIdx.x] = r < rows ? __ldg(a.delta + at0 + r) : 0.f;
    }
    cp_async_wait<1>();
    __syncthreads();
    float s[4][4], dp[4][4];
    dot_tile<D, 4>(sK, sQ, ty, tx, s);
    cp_async_wait<0>();
    __syncthreads();
    dot_tile<D, 4>(sV, sO, ty, tx, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = tx + 8 * j;
        grad_of(s[i][j], dp[i][j], (mine >> i) & 1u, s_lse2[c], s_delta[c], a.scale_log2);
        sP[(ty * 4 + i) * kPad + c] = s[i][j];
      }
    // a thread's rows of P, and then of dS, are read by the eight threads of
    // its own row, all in one warp
    __syncwarp();
    sum_tile<D, 4>(sP, sO, ty, tx, dv);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sP[(ty * 4 + i) * kPad + tx + 8 * j] = dp[i][j];
    __syncwarp();
    sum_tile<D, 4>(sP, sQ, ty, tx, dk);
  }
  cp_async_wait<0>();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = j0 + ty * 4 + i;
    if (j >= a.n_kv) continue;
    if (a.splits > 1) {
      const long long all = (long long)a.B * a.heads_kv * a.n_kv;
      const long long at = ((long long)b * a.heads_kv + hk) * a.n_kv + j;
      put_row<D>(a.part_kv + ((2ll * blockIdx.y) * all + at) * D, dk[i], tx, a.scale);
      put_row<D>(a.part_kv + ((2ll * blockIdx.y + 1) * all + at) * D, dv[i], tx, 1.0f);
    } else {
      put_row<D>(reinterpret_cast<float*>(a.dk.p) + b * a.dk.b + j * a.dk.n + hk * a.dk.h, dk[i], tx, a.scale);
      put_row<D>(reinterpret_cast<float*>(a.dv.p) + b * a.dv.b + j * a.dv.n + hk * a.dv.h, dv[i], tx, 1.0f);
    }
  }
}

template <int D>
cudaError_t run_simt(int which, const CrossArgs& a, cudaStream_t st) {
  constexpr int kRow = row_floats<D>() * (int)sizeof(float);
  const long long rows = (long long)a.group * a.n_q;
  const unsigned row_tiles = (unsigned)((rows + kCrossSimtRows - 1) / kCrossSimtRows);
  const unsigned key_tiles = (unsigned)((a.n_kv + kCrossSimtKvKeys - 1) / kCrossSimtKvKeys), bh = (unsigned)(a.B * a.heads_kv);
  void (*kernel)(CrossArgs);
  int smem;
  unsigned ctas;
  if (which == 0) {
    kernel = cross_simt_forward<D>;
    smem = kCrossSimtRows * kRow + (key_floats<D>() + kKeys * row_floats<D>()) * (int)sizeof(float);
    ctas = row_tiles * bh;
  } else if (which == 1) {
    kernel = cross_simt_dq<D>;
    smem = 2 * kCrossSimtRows * kRow + 2 * key_floats<D>() * (int)sizeof(float);
    ctas = row_tiles * bh;
  } else {
    kernel = cross_simt_dkv<D>;
    smem = 2 * (kCrossSimtKvRows + kCrossSimtKvKeys) * kRow + kCrossSimtKvKeys * kPad * (int)sizeof(float);
    ctas = key_tiles * bh;
  }
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<dim3(ctas, a.splits), kThreads, smem, st>>>(a);
  return cudaGetLastError();
}

cudaError_t run_simt(int which, const CrossArgs& a, int D, cudaStream_t st) {
  return D == 128 ? run_simt<128>(which, a, st) : run_simt<64>(which, a, st);
}

}  // namespace

cudaError_t launch_cross_simt_forward(const CrossArgs& a, int D, cudaStream_t st) { return run_simt(0, a, D, st); }
cudaError_t launch_cross_simt_dq(const CrossArgs& a, int D, cudaStream_t st) { return run_simt(1, a, D, st); }
cudaError_t launch_cross_simt_dkv(const CrossArgs& a, int D, cudaStream_t st) { return run_simt(2, a, D, st); }

}  // namespace bsa
