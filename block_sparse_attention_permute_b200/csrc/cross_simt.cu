// cross_simt.cu — cross attention in fp32 arithmetic (forward, dQ, dK and dV).
//
// With S = scale Q K^T over the attended keys and L = log sum exp S per row:
//   O  = softmax(S) V
//   P  = exp(S - L),  dP = dO V^T,  D = rowsum(dO * O),  dS = P * (dP - D)
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO.
// Tiles of 64 rows by 64 keys, 256 threads as 16 x 16, four by four results
// each; operands in shared memory as fp32 rows padded by 4 floats, so that the
// 16-byte reads of eight consecutive rows fall into different banks.  Bound by
// the FMA pipe (packed fp32 pairs) and the shared-memory reads that feed it.
#include "cross.cuh"

namespace bsa {
namespace {

constexpr int kT = kCrossSimtTile;
constexpr int kPad = kT + 4;     // row stride of a tile of probabilities

template <int D> constexpr int row_floats() { return D + 4; }

// Where row r (of one K/V head's rows) of a per-token tensor starts.
__device__ __forceinline__ float* row_ptr(const CrossArgs& a, const View& v, int b, int hk, long long r) {
  const int g = (int)(r / a.n_q);
  const long long n = r - (long long)g * a.n_q;
  return reinterpret_cast<float*>(v.p) + b * v.b + n * v.n + (long long)(hk * a.group + g) * v.h;
}

__device__ __forceinline__ void put4(float* d, const float* s) {
  *reinterpret_cast<float4*>(d) = __ldg(reinterpret_cast<const float4*>(s));
}
__device__ __forceinline__ void out4(float* d, float4 x) { *reinterpret_cast<float4*>(d) = x; }

// Loads rows r0 .. r0 + 63 (zeros from `end` on) of a row tensor.
template <int D>
__device__ __forceinline__ void load_rows(float* s, const CrossArgs& a, const View& v, int b, int hk, long long r0,
                                          long long end) {
  for (int i = threadIdx.x; i < kT * (D / 4); i += 256) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    float* d = s + r * row_floats<D>() + c;
    if (r0 + r < end) put4(d, row_ptr(a, v, b, hk, r0 + r) + c);
    else *reinterpret_cast<float4*>(d) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

// Loads keys j0 .. j0 + 63 of K or V; keys that are not attended read as zeros
// whatever they hold.
template <int D>
__device__ __forceinline__ void load_keys(float* s, const CrossArgs& a, const View& v, int b, int hk, int j0,
                                          const uint8_t* seen) {
  const float* base = reinterpret_cast<const float*>(v.p) + b * v.b + hk * v.h;
  for (int i = threadIdx.x; i < kT * (D / 4); i += 256) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    float* d = s + r * row_floats<D>() + c;
    if (seen[r]) put4(d, base + (long long)(j0 + r) * v.n + c);
    else *reinterpret_cast<float4*>(d) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

// seen[0..63] of the keys from j0 (all threads; the caller synchronises).
__device__ __forceinline__ void load_seen(uint8_t* seen, const CrossArgs& a, int b, int j0, int keys) {
  if (threadIdx.x < kT) {
    const int j = j0 + threadIdx.x;
    seen[threadIdx.x] = j < keys && (a.key_mask == nullptr || __ldg(a.key_mask + (long long)b * a.n_kv + j) != 0);
  }
}

// acc[i][j] = A row (ty * 4 + i) . B row (tx + 16 j)
template <int D>
__device__ __forceinline__ void dot_tile(const float* A, const float* B, int ty, int tx, float (&acc)[4][4]) {
  float2 s[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int d = 0; d < D; d += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(A + (ty * 4 + i) * row_floats<D>() + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * row_floats<D>() + d);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = fma2(make_float2(x[i].x, x[i].y), make_float2(y[j].x, y[j].y), s[i][j]);
        s[i][j] = fma2(make_float2(x[i].z, x[i].w), make_float2(y[j].z, y[j].w), s[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = s[i][j].x + s[i][j].y;
}

// acc[i][q] += sum_k P[ty * 4 + i][k] B[k][tx * 4 + 64 q ..]
template <int D>
__device__ __forceinline__ void sum_tile(const float* P, const float* B, int ty, int tx, float2 (&acc)[4][D / 32]) {
#pragma unroll 2
  for (int k = 0; k < kT; k += 4) {
    float4 p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(P + (ty * 4 + i) * kPad + k);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
      for (int q = 0; q < D / 64; ++q) {
        const float4 x = *reinterpret_cast<const float4*>(B + (k + kk) * row_floats<D>() + tx * 4 + 64 * q);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float w = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
          acc[i][2 * q] = fma2(make_float2(w, w), make_float2(x.x, x.y), acc[i][2 * q]);
          acc[i][2 * q + 1] = fma2(make_float2(w, w), make_float2(x.z, x.w), acc[i][2 * q + 1]);
        }
      }
    }
  }
}

__device__ __forceinline__ float max16(float x) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float sum16(float x) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <int D>
__device__ __forceinline__ void clear(float2 (&acc)[4][D / 32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int q = 0; q < D / 32; ++q) acc[i][q] = make_float2(0.f, 0.f);
}

// Online softmax over the key tiles of one split; the probabilities replace K
// in shared memory for the product with V.
template <int D>
__global__ void __launch_bounds__(256, 2) cross_simt_forward(CrossArgs a) {
  extern __shared__ float4 smem4[];
  float* sQ = reinterpret_cast<float*>(smem4);
  float* sK = sQ + kT * row_floats<D>();
  float* sV = sK + kT * row_floats<D>();
  __shared__ uint8_t seen[kT];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const long long rows = (long long)a.group * a.n_q;
  const int per = (int)((rows + kT - 1) / kT), bh = blockIdx.x / per;
  const int b = bh / a.heads_kv, hk = bh % a.heads_kv;
  const long long r0 = (long long)(blockIdx.x % per) * kT;
  const int keys = cross_keys(a, b), tiles = (keys + kT - 1) / kT;
  const int t0 = blockIdx.y * a.split_len, t1 = min(tiles, t0 + a.split_len);
  load_rows<D>(sQ, a, a.q, b, hk, r0, rows);
  float m[4], l[4];
  float2 acc[4][D / 32];
  clear<D>(acc);
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = -INFINITY, l[i] = 0.f;
  for (int t = t0; t < t1; ++t) {
    __syncthreads();
    load_seen(seen, a, b, t * kT, keys);
    __syncthreads();
    load_keys<D>(sK, a, a.k, b, hk, t * kT, seen);
    load_keys<D>(sV, a, a.v, b, hk, t * kT, seen);
    __syncthreads();
    float s[4][4];
    dot_tile<D>(sQ, sK, ty, tx, s);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = seen[tx + 16 * j] ? s[i][j] * a.scale_log2 : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
      const float mn = fmaxf(m[i], max16(mx));
      const float base = mn == -INFINITY ? 0.f : mn;
      const float keep = exp2f(m[i] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = exp2f(s[i][j] - base);
        sum += p;
        sK[(ty * 4 + i) * kPad + tx + 16 * j] = p;
      }
      l[i] = l[i] * keep + sum16(sum);
      m[i] = mn;
#pragma unroll
      for (int q = 0; q < D / 32; ++q) acc[i][q] = make_float2(acc[i][q].x * keep, acc[i][q].y * keep);
    }
    __syncthreads();
    sum_tile<D>(sK, sV, ty, tx, acc);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long r = r0 + ty * 4 + i;
    if (r >= rows) continue;
    const long long at = ((long long)b * a.heads + (long long)hk * a.group) * a.n_q + r;
    if (a.splits > 1) {
      const long long p = blockIdx.y * cross_rows(a) + at;
#pragma unroll
      for (int q = 0; q < D / 64; ++q)
        out4(a.part_o + p * D + tx * 4 + 64 * q,
             make_float4(acc[i][2 * q].x, acc[i][2 * q].y, acc[i][2 * q + 1].x, acc[i][2 * q + 1].y));
      if (tx == 0) a.part_ml[p] = make_float2(m[i], l[i]);
    } else {
      const float inv = m[i] == -INFINITY ? 0.f : 1.f / l[i];
      float* d = row_ptr(a, a.o, b, hk, r);
#pragma unroll
      for (int q = 0; q < D / 64; ++q)
        out4(d + tx * 4 + 64 * q, make_float4(acc[i][2 * q].x * inv, acc[i][2 * q].y * inv,
                                              acc[i][2 * q + 1].x * inv, acc[i][2 * q + 1].y * inv));
      if (tx == 0 && a.lse) a.lse[at] = (m[i] + log2f(l[i])) * 0.69314718055994531f;
    }
  }
}

// P and dS of one tile: s holds Q.K on entry and P on return, dp holds dO.V on
// entry and dS / scale on return.  Rows of the tile are (i), keys (j) if ROWS,
// the other way round else; lse2 is in log2 units, +inf where P is 0.
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
__global__ void __launch_bounds__(256) cross_simt_dq(CrossArgs a) {
  extern __shared__ float4 smem4[];
  float* sQ = reinterpret_cast<float*>(smem4);
  float* sO = sQ + kT * row_floats<D>();
  float* sK = sO + kT * row_floats<D>();
  float* sV = sK + kT * row_floats<D>();
  __shared__ uint8_t seen[kT];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const long long rows = (long long)a.group * a.n_q;
  const int per = (int)((rows + kT - 1) / kT), bh = blockIdx.x / per;
  const int b = bh / a.heads_kv, hk = bh % a.heads_kv;
  const long long r0 = (long long)(blockIdx.x % per) * kT;
  const long long at0 = ((long long)b * a.heads + (long long)hk * a.group) * a.n_q;
  const int keys = cross_keys(a, b), tiles = (keys + kT - 1) / kT;
  load_rows<D>(sQ, a, a.q, b, hk, r0, rows);
  load_rows<D>(sO, a, a.d_o, b, hk, r0, rows);
  float lse2[4], delta[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long r = r0 + ty * 4 + i;
    lse2[i] = lse2_of(a, at0 + r, r < rows);
    delta[i] = r < rows ? __ldg(a.delta + at0 + r) : 0.f;
  }
  float2 acc[4][D / 32];
  clear<D>(acc);
  const int t0 = blockIdx.y * a.split_len, t1 = min(tiles, t0 + a.split_len);
  for (int t = t0; t < t1; ++t) {
    __syncthreads();
    load_seen(seen, a, b, t * kT, keys);
    __syncthreads();
    load_keys<D>(sK, a, a.k, b, hk, t * kT, seen);
    load_keys<D>(sV, a, a.v, b, hk, t * kT, seen);
    __syncthreads();
    float s[4][4], dp[4][4];
    dot_tile<D>(sQ, sK, ty, tx, s);
    dot_tile<D>(sO, sV, ty, tx, dp);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        grad_of(s[i][j], dp[i][j], seen[tx + 16 * j], lse2[i], delta[i], a.scale_log2);
        sV[(ty * 4 + i) * kPad + tx + 16 * j] = dp[i][j];
      }
    __syncthreads();
    sum_tile<D>(sV, sK, ty, tx, acc);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long r = r0 + ty * 4 + i;
    if (r >= rows) continue;
    float* d = a.splits > 1 ? a.part_o + (blockIdx.y * cross_rows(a) + at0 + r) * D : row_ptr(a, a.dq, b, hk, r);
#pragma unroll
    for (int q = 0; q < D / 64; ++q)
      out4(d + tx * 4 + 64 * q, make_float4(acc[i][2 * q].x * a.scale, acc[i][2 * q].y * a.scale,
                                            acc[i][2 * q + 1].x * a.scale, acc[i][2 * q + 1].y * a.scale));
  }
}

// dK and dV of 64 keys, over the row tiles of one split.
template <int D>
__global__ void __launch_bounds__(256) cross_simt_dkv(CrossArgs a) {
  extern __shared__ float4 smem4[];
  float* sK = reinterpret_cast<float*>(smem4);
  float* sV = sK + kT * row_floats<D>();
  float* sQ = sV + kT * row_floats<D>();
  float* sO = sQ + kT * row_floats<D>();
  float* sP = sO + kT * row_floats<D>();
  float* sS = sP + kT * kPad;
  __shared__ uint8_t seen[kT];
  __shared__ float s_lse2[kT], s_delta[kT];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int per = (a.n_kv + kT - 1) / kT, bh = blockIdx.x / per;
  const int b = bh / a.heads_kv, hk = bh % a.heads_kv;
  const int j0 = (int)(blockIdx.x % per) * kT;
  const long long rows = (long long)a.group * a.n_q;
  const long long at0 = ((long long)b * a.heads + (long long)hk * a.group) * a.n_q;
  const int keys = cross_keys(a, b);
  const long long t0 = (long long)blockIdx.y * a.split_len;
  long long t1 = min((rows + kT - 1) / kT, t0 + a.split_len);
  if (j0 >= keys) t1 = t0;      // no key of this tile is attended
  load_seen(seen, a, b, j0, keys);
  __syncthreads();
  load_keys<D>(sK, a, a.k, b, hk, j0, seen);
  load_keys<D>(sV, a, a.v, b, hk, j0, seen);
  float2 dk[4][D / 32], dv[4][D / 32];
  clear<D>(dk);
  clear<D>(dv);
  for (long long t = t0; t < t1; ++t) {
    __syncthreads();
    load_rows<D>(sQ, a, a.q, b, hk, t * kT, rows);
    load_rows<D>(sO, a, a.d_o, b, hk, t * kT, rows);
    if (threadIdx.x < kT) {
      const long long r = t * kT + threadIdx.x;
      s_lse2[threadIdx.x] = lse2_of(a, at0 + r, r < rows);
      s_delta[threadIdx.x] = r < rows ? __ldg(a.delta + at0 + r) : 0.f;
    }
    __syncthreads();
    float s[4][4], dp[4][4];
    dot_tile<D>(sK, sQ, ty, tx, s);
    dot_tile<D>(sV, sO, ty, tx, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = tx + 16 * j;
        grad_of(s[i][j], dp[i][j], seen[ty * 4 + i], s_lse2[c], s_delta[c], a.scale_log2);
        sP[(ty * 4 + i) * kPad + c] = s[i][j];
        sS[(ty * 4 + i) * kPad + c] = dp[i][j];
      }
    __syncthreads();
    sum_tile<D>(sP, sO, ty, tx, dv);
    sum_tile<D>(sS, sQ, ty, tx, dk);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = j0 + ty * 4 + i;
    if (j >= a.n_kv) continue;
#pragma unroll
    for (int q = 0; q < D / 64; ++q) {
      const int c = tx * 4 + 64 * q;
      const float4 gk = make_float4(dk[i][2 * q].x * a.scale, dk[i][2 * q].y * a.scale, dk[i][2 * q + 1].x * a.scale,
                                    dk[i][2 * q + 1].y * a.scale);
      const float4 gv = make_float4(dv[i][2 * q].x, dv[i][2 * q].y, dv[i][2 * q + 1].x, dv[i][2 * q + 1].y);
      if (a.splits > 1) {
        const long long all = (long long)a.B * a.heads_kv * a.n_kv;
        const long long at = ((long long)b * a.heads_kv + hk) * a.n_kv + j;
        out4(a.part_kv + ((2ll * blockIdx.y) * all + at) * D + c, gk);
        out4(a.part_kv + ((2ll * blockIdx.y + 1) * all + at) * D + c, gv);
      } else {
        out4(reinterpret_cast<float*>(a.dk.p) + b * a.dk.b + j * a.dk.n + hk * a.dk.h + c, gk);
        out4(reinterpret_cast<float*>(a.dv.p) + b * a.dv.b + j * a.dv.n + hk * a.dv.h + c, gv);
      }
    }
  }
}

template <int D>
cudaError_t run_simt(int which, const CrossArgs& a, cudaStream_t st) {
  const int tile = kT * row_floats<D>() * (int)sizeof(float);
  const long long rows = (long long)a.group * a.n_q;
  const unsigned row_tiles = (unsigned)((rows + kT - 1) / kT), key_tiles = (unsigned)((a.n_kv + kT - 1) / kT);
  void (*kernel)(CrossArgs);
  int smem;
  dim3 grid;
  if (which == 0) {
    kernel = cross_simt_forward<D>;
    smem = 3 * tile;
    grid = dim3(row_tiles * a.B * a.heads_kv, a.splits);
  } else if (which == 1) {
    kernel = cross_simt_dq<D>;
    smem = 4 * tile;
    grid = dim3(row_tiles * a.B * a.heads_kv, a.splits);
  } else {
    kernel = cross_simt_dkv<D>;
    smem = 4 * tile + 2 * kT * kPad * (int)sizeof(float);
    grid = dim3(key_tiles * a.B * a.heads_kv, a.splits);
  }
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, 256, smem, st>>>(a);
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
