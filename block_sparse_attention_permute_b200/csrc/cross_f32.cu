// cross_f32.cu — cross attention of fp32 tensors (forward, dQ, dK and dV).
//
// With S = scale Q K^T over the attended keys and L = log sum exp S per row:
//   O  = softmax(S) V
//   P  = exp(S - L),  dP = dO V^T,  D = rowsum(dO * O),  dS = P * (dP - D)
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO.
// Products run on the tensor cores in tf32, three for one: with x = h + l, h the 11
// leading bits that tf32 keeps, a b = ha hb + ha lb + la hb up to 1.75 2^-20 of its
// size (la lb below 2^-20, and of each l the 2 of 13 bits that tf32 drops, 0.75 2^-21
// for either; all short of the product, 0.27 2^-20 on average), every sum in fp32.
// As the tensor core rounds each addition toward zero, a tile's products are summed
// from zero, the small ones apart from the large, and joined to the running sum by
// fp32 additions.  The
// legacy warp MMA serves here: tcgen05 would want both parts of both operands in
// shared memory, 256 KB for one pair of 128 x 128 tiles.  A warp owns 16 rows of
// the result (query rows; keys for dK and dV) and keeps its logits, probabilities
// and sums in registers: the columns 2t and 2t + 1 that a thread holds of eight
// logits become the operand's columns t and t + 4, and the other operand's rows are
// taken in the same order.  Rows in shared memory are padded by 4 floats, so that
// ldmatrix (eight rows, 16 bytes each) and the loads of rows 2t, columns g both
// touch all banks once.  Two or three CTAs of 64 rows (or keys) share an SM and cover
// one another's loads and barriers.
//
// Measured on B200, 1560 rows x 226 keys x 12 heads of 128: forward 77 us, dQ 102 us,
// dK and dV 125 us (28 to 35 TFLOP/s of fp32 products), a training step 319 us; packed
// fp32 FMAs took 404 us (bound by 3.1 shared-memory wavefronts per 16-byte load), a
// library's fp32 products with the rest in torch 387 us.  Bound by the latency of
// dependent instructions (load, split, MMA) with 7 or 8 warps on an SM: the tensor
// pipe is 44 to 50% busy, issue slots 32 to 38%; and by 300 CTAs for 296 (dQ) or 444
// (forward) places, and 288.
#include "cross.cuh"

namespace bsa {
namespace {

constexpr int kThreads = 128;
constexpr int kKeys = kCrossF32Keys, kRows = kCrossF32Rows;

template <int D> constexpr int row_floats() { return D + 4; }

// Where row r (of one K/V head's rows) of a per-token tensor starts.
__device__ __forceinline__ float* row_ptr(const CrossArgs& a, const View& v, int b, int hk, long long r) {
  const int g = (int)(r / a.n_q);
  const long long n = r - (long long)g * a.n_q;
  return reinterpret_cast<float*>(v.p) + b * v.b + n * v.n + (long long)(hk * a.group + g) * v.h;
}

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
  for (int i = threadIdx.x; i < 32 * kPer; i += kThreads) {
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

// x = hi + lo, hi the 11 leading bits that tf32 keeps.
__device__ __forceinline__ void split(uint32_t x, uint32_t& hi, uint32_t& lo) {
  hi = x & 0xffffe000u;
  lo = __float_as_uint(__uint_as_float(x) - __uint_as_float(hi));
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// c += a b, 16 x 8 x 8, tf32 operands.
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// c + small += a b for operands given as fp32.
struct Split4 {
  uint32_t hi[4], lo[4];
};
__device__ __forceinline__ Split4 split4(const uint32_t (&x)[4]) {
  Split4 s;
#pragma unroll
  for (int i = 0; i < 4; ++i) split(x[i], s.hi[i], s.lo[i]);
  return s;
}
__device__ __forceinline__ void mma3(float (&c)[4], float (&small)[4], const Split4& a, uint32_t b0, uint32_t b1) {
  uint32_t h0, l0, h1, l1;
  split(b0, h0, l0);
  split(b1, h1, l1);
  mma_tf32(small, a.lo, h0, h1);
  mma_tf32(small, a.hi, l0, l1);
  mma_tf32(c, a.hi, h0, h1);
}

// s[j] = the 16 rows of A times rows 8 j .. 8 j + 7 of B, contracted over D.  Lane
// (g, t) = (lane / 4, lane % 4) holds of s[j] row g columns 2t, 2t + 1 and row g + 8
// the same columns.
template <int D>
__device__ __forceinline__ void dot_tile(const float* A, const float* B, int lane, float (&s)[4][4]) {
  float small[4][4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[j][i] = small[j][i] = 0.f;
  // ldmatrix: lanes 8 m .. 8 m + 7 give the rows of matrix m
  const uint32_t pa = smem_addr(A + (lane & 15) * row_floats<D>() + (lane >> 4) * 4);
  const uint32_t pb = smem_addr(B + ((lane & 7) + (lane >> 4) * 8) * row_floats<D>() + ((lane >> 3) & 1) * 4);
#pragma unroll 4
  for (int k = 0; k < D; k += 8) {
    uint32_t x[4];
    ldmatrix4(x, pa + k * 4);
    const Split4 xa = split4(x);
#pragma unroll
    for (int jj = 0; jj < 2; ++jj) {
      uint32_t y[4];
      ldmatrix4(y, pb + (jj * 16 * row_floats<D>() + k) * 4);
      mma3(s[2 * jj], small[2 * jj], xa, y[0], y[1]);
      mma3(s[2 * jj + 1], small[2 * jj + 1], xa, y[2], y[3]);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[j][i] += small[j][i];
}

// acc[n] += P (16 rows, 32 columns held as dot_tile leaves them) times the 32 rows
// of B, columns 8 n .. 8 n + 7.  The tile's products start from zero and join acc
// by an fp32 addition to nearest: carried from tile to tile in the MMA, whose
// additions all round toward zero, a sum of terms of one sign lost 2.4e-4 of itself
// over 32 768 rows.
template <int D>
__device__ __forceinline__ void sum_tile(const float (&p)[4][4], const float* B, int lane, float (&acc)[D / 8][4]) {
  const float* q = B + 2 * (lane & 3) * row_floats<D>() + (lane >> 2);
  Split4 x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t y[4] = {__float_as_uint(p[j][0]), __float_as_uint(p[j][2]), __float_as_uint(p[j][1]),
                           __float_as_uint(p[j][3])};
    x[j] = split4(y);
  }
#pragma unroll
  for (int n = 0; n < D / 8; ++n) {
    float large[4] = {0.f, 0.f, 0.f, 0.f}, small[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float* b = q + 8 * j * row_floats<D>() + 8 * n;
      mma3(large, small, x[j], __float_as_uint(b[0]), __float_as_uint(b[row_floats<D>()]));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] += large[i] + small[i];
  }
}

// Over the four threads of a row.
__device__ __forceinline__ float max_row(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float sum_row(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

template <int N>
__device__ __forceinline__ void clear(float (&acc)[N][4]) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
}

// Row g (half 0) or g + 8 (half 1) of acc, times `by`.
template <int D>
__device__ __forceinline__ void put_row(float* d, const float (&acc)[D / 8][4], int half, int lane, float by) {
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
    *reinterpret_cast<float2*>(d + 8 * n + 2 * (lane & 3)) = make_float2(acc[n][2 * half] * by, acc[n][2 * half + 1] * by);
}

// Column of a 32-column tile that element i of s[j] stands for.
__device__ __forceinline__ int column(int j, int i, int lane) { return 8 * j + 2 * (lane & 3) + (i & 1); }

// Online softmax over the key tiles of one split.
template <int D>
__global__ void __launch_bounds__(kThreads, 3) cross_f32_forward(CrossArgs a) {
  extern __shared__ float4 smem4[];
  float* sQ = reinterpret_cast<float*>(smem4);
  float* sK = sQ + kRows * row_floats<D>();
  float* sV = sK + kKeys * row_floats<D>();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long rows = (long long)a.group * a.n_q;
  const int per = (int)((rows + kRows - 1) / kRows), bh = blockIdx.x / per;
  const int b = bh / a.heads_kv, hk = bh % a.heads_kv;
  const long long r0 = (long long)(blockIdx.x % per) * kRows;
  const int keys = cross_keys(a, b), tiles = (keys + kKeys - 1) / kKeys;
  const int t0 = blockIdx.y * a.split_len, t1 = min(tiles, t0 + a.split_len);
  load_rows<D, kRows>(sQ, a, a.q, b, hk, r0, rows);
  const bool busy = r0 + 16 * warp < rows;       // the warp has rows
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float acc[D / 8][4];
  clear(acc);
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
    if (busy) {
      dot_tile<D>(sQ + 16 * warp * row_floats<D>(), sK, lane, s);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 2 * h; i < 2 * h + 2; ++i) {
            s[j][i] = (seen >> column(j, i, lane)) & 1u ? s[j][i] * a.scale_log2 : -INFINITY;
            mx = fmaxf(mx, s[j][i]);
          }
        const float mn = fmaxf(m[h], max_row(mx));
        const float base = mn == -INFINITY ? 0.f : mn;
        const float keep = exp2f(m[h] - base);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 2 * h; i < 2 * h + 2; ++i) {
            s[j][i] = exp2f(s[j][i] - base);
            sum += s[j][i];
          }
        l[h] = l[h] * keep + sum_row(sum);
        m[h] = mn;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) acc[n][2 * h] *= keep, acc[n][2 * h + 1] *= keep;
      }
    }
    cp_async_wait<0>();
    __syncthreads();
    if (busy) sum_tile<D>(s, sV, lane, acc);
  }
  cp_async_wait<0>();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const long long r = r0 + 16 * warp + 8 * h + (lane >> 2);
    if (r >= rows) continue;
    const long long at = ((long long)b * a.heads + (long long)hk * a.group) * a.n_q + r;
    if (a.splits > 1) {
      const long long p = blockIdx.y * cross_rows(a) + at;
      put_row<D>(a.part_o + p * D, acc, h, lane, 1.0f);
      if ((lane & 3) == 0) a.part_ml[p] = make_float2(m[h], l[h]);
    } else {
      put_row<D>(row_ptr(a, a.o, b, hk, r), acc, h, lane, m[h] == -INFINITY ? 0.f : 1.f / l[h]);
      if ((lane & 3) == 0 && a.lse) a.lse[at] = (m[h] + log2f(l[h])) * 0.69314718055994531f;
    }
  }
}

// P and dS of one logit: s holds Q.K on entry, dp holds dO.V on entry and dS /
// scale on return.  lse2 is in log2 units, +inf where P is 0.
__device__ __forceinline__ void grad_of(float& s, float& dp, bool seen, float lse2, float delta, float scale_log2) {
  s = seen ? exp2f(fmaf(s, scale_log2, -lse2)) : 0.f;
  dp = seen ? s * (dp - delta) : 0.f;
}

__device__ __forceinline__ float lse2_of(const CrossArgs& a, long long at, bool in) {
  const float x = in ? __ldg(a.lse + at) : -INFINITY;
  return x == -INFINITY ? INFINITY : x * 1.4426950408889634f;
}

// dQ of 64 rows, over the key tiles of one split.
template <int D>
__global__ void __launch_bounds__(kThreads, 2) cross_f32_dq(CrossArgs a) {
  extern __shared__ float4 smem4[];
  float* sQ = reinterpret_cast<float*>(smem4);
  float* sO = sQ + kRows * row_floats<D>();
  float* sK = sO + kRows * row_floats<D>();
  float* sV = sK + kKeys * row_floats<D>();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long rows = (long long)a.group * a.n_q;
  const int per = (int)((rows + kRows - 1) / kRows), bh = blockIdx.x / per;
  const int b = bh / a.heads_kv, hk = bh % a.heads_kv;
  const long long r0 = (long long)(blockIdx.x % per) * kRows;
  const long long at0 = ((long long)b * a.heads + (long long)hk * a.group) * a.n_q;
  const int keys = cross_keys(a, b), tiles = (keys + kKeys - 1) / kKeys;
  load_rows<D, kRows>(sQ, a, a.q, b, hk, r0, rows);
  load_rows<D, kRows>(sO, a, a.d_o, b, hk, r0, rows);
  const bool busy = r0 + 16 * warp < rows;
  float lse2[2], delta[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const long long r = r0 + 16 * warp + 8 * h + (lane >> 2);
    lse2[h] = lse2_of(a, at0 + r, r < rows);
    delta[h] = r < rows ? __ldg(a.delta + at0 + r) : 0.f;
  }
  float acc[D / 8][4];
  clear(acc);
  const bool one = one_key(a, b, keys);          // dS is 0
  const int t0 = blockIdx.y * a.split_len, t1 = one ? 0 : min(tiles, t0 + a.split_len);
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
    if (busy) dot_tile<D>(sQ + 16 * warp * row_floats<D>(), sK, lane, s);
    cp_async_wait<0>();
    __syncthreads();
    if (busy) {
      dot_tile<D>(sO + 16 * warp * row_floats<D>(), sV, lane, dp);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          grad_of(s[j][i], dp[j][i], (seen >> column(j, i, lane)) & 1u, lse2[i >> 1], delta[i >> 1], a.scale_log2);
      sum_tile<D>(dp, sK, lane, acc);
    }
  }
  cp_async_wait<0>();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const long long r = r0 + 16 * warp + 8 * h + (lane >> 2);
    if (r >= rows) continue;
    put_row<D>(a.splits > 1 ? a.part_o + (blockIdx.y * cross_rows(a) + at0 + r) * D : row_ptr(a, a.dq, b, hk, r), acc, h,
               lane, a.scale);
  }
}

// dK and dV of 64 keys, over the tiles of 32 rows of one split.
template <int D>
__global__ void __launch_bounds__(kThreads, 2) cross_f32_dkv(CrossArgs a) {
  constexpr int R = kCrossF32KvRows, kN = kCrossF32KvKeys;
  extern __shared__ float4 smem4[];
  float* sK = reinterpret_cast<float*>(smem4);
  float* sV = sK + kN * row_floats<D>();
  float* sQ = sV + kN * row_floats<D>();
  float* sO = sQ + R * row_floats<D>();
  __shared__ float s_lse2[R], s_delta[R];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
  const uint32_t seen = (warp >= 2 ? seen1 : seen0) >> (16 * (warp & 1)) & 0xffffu;   // the warp's 16 keys
  const bool one = one_key(a, b, keys);          // dS is 0
  float dk[D / 8][4], dv[D / 8][4];
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
    if (seen) dot_tile<D>(sK + 16 * warp * row_floats<D>(), sQ, lane, s);
    cp_async_wait<0>();
    __syncthreads();
    if (seen) {
      dot_tile<D>(sV + 16 * warp * row_floats<D>(), sO, lane, dp);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = column(j, i, lane);
          grad_of(s[j][i], dp[j][i], (seen >> ((lane >> 2) + 8 * (i >> 1))) & 1u, s_lse2[c], s_delta[c], a.scale_log2);
        }
      sum_tile<D>(s, sO, lane, dv);
      if (!one) sum_tile<D>(dp, sQ, lane, dk);
    }
  }
  cp_async_wait<0>();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = j0 + 16 * warp + 8 * h + (lane >> 2);
    if (j >= a.n_kv) continue;
    if (a.splits > 1 || a.slot_of) {
      const long long all = (long long)a.B * a.heads_kv * a.n_kv;
      const long long at = ((long long)b * a.heads_kv + hk) * a.n_kv + j;
      put_row<D>(a.part_kv + ((2ll * blockIdx.y) * all + at) * D, dk, h, lane, a.scale);
      put_row<D>(a.part_kv + ((2ll * blockIdx.y + 1) * all + at) * D, dv, h, lane, 1.0f);
    } else {
      put_row<D>(reinterpret_cast<float*>(a.dk.p) + b * a.dk.b + j * a.dk.n + hk * a.dk.h, dk, h, lane, a.scale);
      put_row<D>(reinterpret_cast<float*>(a.dv.p) + b * a.dv.b + j * a.dv.n + hk * a.dv.h, dv, h, lane, 1.0f);
    }
  }
}

// The forward (0), dQ (1), or dK and dV (2).
template <int D>
struct F32 {
  static auto kernel(int which) {
    return which == 0 ? cross_f32_forward<D> : which == 1 ? cross_f32_dq<D> : cross_f32_dkv<D>;
  }
  static int smem(int which) {
    return row_floats<D>() * (int)sizeof(float) *
           (which == 0 ? kRows + 2 * kKeys : 2 * (which == 1 ? kRows + kKeys : kCrossF32KvRows + kCrossF32KvKeys));
  }
  static cudaError_t run(int which, const CrossArgs& a, cudaStream_t st) {
    const long long rows = (long long)a.group * a.n_q;
    const unsigned row_tiles = (unsigned)((rows + kRows - 1) / kRows), bh = (unsigned)(a.B * a.heads_kv);
    const unsigned key_tiles = (unsigned)((a.n_kv + kCrossF32KvKeys - 1) / kCrossF32KvKeys);
    kernel(which)<<<dim3((which == 2 ? key_tiles : row_tiles) * bh, a.splits), kThreads, smem(which), st>>>(a);
    return cudaGetLastError();
  }
  static cudaError_t prepare() {
    for (int which = 0; which < 3; ++which) {
      const cudaError_t e = cudaFuncSetAttribute(kernel(which), cudaFuncAttributeMaxDynamicSharedMemorySize, smem(which));
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
};

cudaError_t run_f32(int which, const CrossArgs& a, int D, cudaStream_t st) {
  return D == 128 ? F32<128>::run(which, a, st) : F32<64>::run(which, a, st);
}

}  // namespace

cudaError_t prepare_cross_f32(int D) { return D == 128 ? F32<128>::prepare() : F32<64>::prepare(); }
cudaError_t launch_cross_f32_forward(const CrossArgs& a, int D, cudaStream_t st) { return run_f32(0, a, D, st); }
cudaError_t launch_cross_f32_dq(const CrossArgs& a, int D, cudaStream_t st) { return run_f32(1, a, D, st); }
cudaError_t launch_cross_f32_dkv(const CrossArgs& a, int D, cudaStream_t st) { return run_f32(2, a, D, st); }

}  // namespace bsa
