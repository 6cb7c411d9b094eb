// rotary.cu — rotary positions over the latent grid (bsa_rope_*, bsa_rotary).
//
// A rotated pair (a, b) of a head becomes mscale (a cos w - b sin w,
// a sin w + b cos w) with w = pos f, pos the token's t, y or x and f the
// pair's frequency.  The map is linear and its transpose turns by -w, so the
// backward pass is the same kernel with the sine negated.
#include <cfloat>
#include <cmath>
#include <cstring>
#include <new>

#include "bsa.h"
#include "kernels.cuh"
#include "views.cuh"

struct bsa_rope_s {
  Geo g;
  int is_bf16;
  int device;
  int heads_k;
  int layout;
  int pairs[3];        // per axis
  double turns[64];    // f / (2 pi) of every pair
  float mscale;
};

namespace bsa {

struct RotaryArgs {
  View in[2], out[2];      // Q, K (K.p = null: none)
  int heads[2];
  int in_place[2];
  long long rows;          // B * n_tot
  long long n_video;
  FastDiv div_tot, div_w, div_h;
  int pt, pty, pairs;      // pairs of the t axis, of t and y, of all axes
  int log_units;           // threads per token
  int heads_per_cta;       // heads (of Q then K) each CTA row takes
  float sine_sign, mscale;
  const int64_t* t_origin;
  double turns[64];
};

template <int BYTES> struct Chunk;
template <> struct Chunk<16> { using type = uint4; };
template <> struct Chunk<8> { using type = uint2; };
template <> struct Chunk<4> { using type = uint32_t; };
template <> struct Chunk<2> { using type = uint16_t; };

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& d, float x) { d = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }

// One thread takes the same V elements (interleaved) or the same V pairs, V
// elements at a time (half), of every head of a token, so that its angles are
// formed once: the turn pos f / (2 pi) is reduced to [-1/2, 1/2] in double
// (off by 4 2^-53 of itself: 2^-21 radians at position 2^30, where the range
// ends) and only then goes to fp32.
// Bound by memory: every element is read and written once, in V-element
// accesses (16 bytes where the layout allows), consecutive threads on
// consecutive parts of a token's head.  Measured on B200: HunyuanVideo's Q and
// K (57 856 tokens, 24 heads of 128, bf16) 220 us, 6.46 TB/s; Wan2.1-1.3B's
// out of a fused projection (32 760 tokens, 12 heads) 67 us, 5.98 TB/s; half
// layout, 131 040 tokens of 12 heads 249 us, 6.46 TB/s; half layout whose halves
// are 63 elements (2-byte accesses) 88 us instead of 66.
template <typename T, bool HALF, int V>
__global__ void __launch_bounds__(256) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  constexpr int P = HALF ? V : V / 2;          // pairs per thread
  constexpr int kBatch = 4;                    // heads in flight per thread
  using C = typename Chunk<V * sizeof(T)>::type;
  __shared__ double s_turns[64];
  if (threadIdx.x < 64) s_turns[threadIdx.x] = a.turns[threadIdx.x];
  __syncthreads();
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long row = id >> a.log_units;
  if (row >= a.rows) return;
  const int unit = (int)id & ((1 << a.log_units) - 1);
  const int b = (int)fdiv((uint32_t)row, a.div_tot);
  const int n = (int)(row - (long long)b * a.div_tot.d);
  bool turned = n < a.n_video;
  int e0, e1 = 0, p0;                          // first element(s), first pair
  if constexpr (HALF) {
    const int units = a.pairs / V;             // units that hold pairs; the rest pass two chunks through
    if (unit < units) {
      p0 = unit * V;
      e0 = p0;
      e1 = p0 + a.pairs;
    } else {
      turned = false;
      p0 = 0;
      e0 = 2 * unit * V;
      e1 = e0 + V;
    }
  } else {
    e0 = unit * V;
    p0 = unit * P;
    turned = turned && p0 < a.pairs;
  }
  float cs[P], sn[P];
  if (turned) {
    const uint32_t q = fdiv((uint32_t)n, a.div_w), t = fdiv(q, a.div_h);
    const double px = (double)(n - q * a.div_w.d), py = (double)(q - t * a.div_h.d);
    const double pt = (double)((a.t_origin ? __ldg(reinterpret_cast<const long long*>(a.t_origin) + b) : 0ll) + t);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int p = min(p0 + i, a.pairs - 1);
      const double w = (p < a.pt ? pt : p < a.pty ? py : px) * s_turns[p];
      float s, c;
      sincospif(2.0f * (float)(w - rint(w)), &s, &c);
      cs[i] = c * a.mscale;
      sn[i] = s * a.sine_sign;
    }
  }
  const int j0 = blockIdx.y * a.heads_per_cta, j1 = j0 + a.heads_per_cta;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (which == 1 && a.in[1].p == nullptr) break;
    if (!turned && a.in_place[which]) continue;
    const int h0 = which ? max(j0 - a.heads[0], 0) : j0;
    const int h1 = which ? min(j1 - a.heads[0], a.heads[1]) : min(j1, a.heads[0]);
    const View vi = a.in[which], vo = a.out[which];
    const T* src = reinterpret_cast<const T*>(vi.p) + b * vi.b + n * vi.n;
    T* dst = reinterpret_cast<T*>(vo.p) + b * vo.b + n * vo.n;
    // kBatch heads are read before the first of them is written (a store may
    // alias any later load as far as the compiler knows).
    for (int hb = h0; hb < h1; hb += kBatch) {
      union Part { C raw; T v[V]; } x[kBatch], y[HALF ? kBatch : 1];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (hb + u >= h1) break;
        const T* s = src + (hb + u) * vi.h;
        x[u].raw = *reinterpret_cast<const C*>(s + e0);
        if constexpr (HALF) y[u].raw = *reinterpret_cast<const C*>(s + e1);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (hb + u >= h1) break;
        T* d = dst + (hb + u) * vo.h;
        if constexpr (HALF) {
          if (turned) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float f = to_f(x[u].v[i]), g = to_f(y[u].v[i]);
              from_f(x[u].v[i], f * cs[i] - g * sn[i]);
              from_f(y[u].v[i], f * sn[i] + g * cs[i]);
            }
          }
          *reinterpret_cast<C*>(d + e1) = y[u].raw;
        } else if (turned) {
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const float f = to_f(x[u].v[2 * i]), g = to_f(x[u].v[2 * i + 1]);
            if (p0 + i < a.pairs) {            // elements past R keep their bits
              from_f(x[u].v[2 * i], f * cs[i] - g * sn[i]);
              from_f(x[u].v[2 * i + 1], f * sn[i] + g * cs[i]);
            }
          }
        }
        *reinterpret_cast<C*>(d + e0) = x[u].raw;
      }
    }
  }
}

template <typename T, bool HALF, int V>
static cudaError_t launch_rotary_t(const Geo& g, RotaryArgs& a, cudaStream_t st) {
  const int units = g.D / (HALF ? 2 * V : V);
  a.log_units = 0;
  while ((1 << a.log_units) < units) ++a.log_units;
  const long long threads = a.rows * units;
  const int heads = a.heads[0] + (a.in[1].p ? a.heads[1] : 0);
  // One thread per unit walks all heads when the tokens alone fill the GPU
  // (148 SMs of 1024 threads); otherwise the heads are split over CTA rows.
  const long long want = (148ll * 1024 + threads - 1) / threads;
  const int split = (int)(want < 1 ? 1 : want > heads ? heads : want);
  a.heads_per_cta = (heads + split - 1) / split;
  const dim3 grid((unsigned)((threads + 255) / 256), (unsigned)((heads + a.heads_per_cta - 1) / a.heads_per_cta));
  rotary_kernel<T, HALF, V><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
static cudaError_t launch_rotary(const Geo& g, bool half, RotaryArgs& a, cudaStream_t st) {
  constexpr int kFull = 16 / sizeof(T);
  if (!half) return launch_rotary_t<T, false, kFull>(g, a, st);
  // the halves start R / 2 elements apart: the widest access that divides it
  if (a.pairs % kFull == 0) return launch_rotary_t<T, true, kFull>(g, a, st);
  if constexpr (kFull == 8)
    if (a.pairs % 4 == 0) return launch_rotary_t<T, true, 4>(g, a, st);
  if (a.pairs % 2 == 0) return launch_rotary_t<T, true, 2>(g, a, st);
  return launch_rotary_t<T, true, 1>(g, a, st);
}

}  // namespace bsa

extern "C" {

bsa_status bsa_rope_create(bsa_rope_t* out, bsa_plan_t plan, const bsa_rope_config_t* c) {
  if (out == nullptr) return bsa_internal_fail(BSA_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (c == nullptr) return bsa_internal_fail(BSA_ERR_INVALID_ARG, "rope config is NULL");
  int R = 0;
  for (int x = 0; x < 3; ++x) {
    if (c->dim[x] < 0 || (c->dim[x] & 1) || c->dim[x] > 128)
      return bsa_internal_fail(BSA_ERR_INVALID_ARG, "rope dim of each axis must be even, in [0, head_dim]");
    R += c->dim[x];
  }
  if (c->layout != BSA_ROPE_INTERLEAVED && c->layout != BSA_ROPE_HALF)
    return bsa_internal_fail(BSA_ERR_INVALID_ARG, "bad rope layout");
  if (c->scaling < BSA_ROPE_NONE || c->scaling > BSA_ROPE_YARN)
    return bsa_internal_fail(BSA_ERR_INVALID_ARG, "bad rope scaling");
  if (!(c->theta > 1.0) || !std::isfinite(c->theta))
    return bsa_internal_fail(BSA_ERR_INVALID_ARG, "rope theta must be above 1");
  if (!(c->mscale >= FLT_MIN) || !(c->mscale <= FLT_MAX))
    return bsa_internal_fail(BSA_ERR_INVALID_ARG, "rope mscale must be above 0 and a normal number in fp32");
  for (int x = 0; x < 3; ++x) {
    if (c->scaling != BSA_ROPE_NONE && (!(c->factor[x] >= 1.0) || !std::isfinite(c->factor[x])))
      return bsa_internal_fail(BSA_ERR_INVALID_ARG, "rope factor must be at least 1");
    if (c->scaling == BSA_ROPE_YARN && (!(c->orig_len[x] > 0.0) || !std::isfinite(c->orig_len[x])))
      return bsa_internal_fail(BSA_ERR_INVALID_ARG, "rope orig_len must be above 0");
  }
  if (c->scaling == BSA_ROPE_YARN &&
      (!(c->beta_slow >= 0.0) || !(c->beta_fast > c->beta_slow) || !std::isfinite(c->beta_fast)))
    return bsa_internal_fail(BSA_ERR_INVALID_ARG, "rope needs beta_fast > beta_slow >= 0");
  if (c->heads_k < 0 || c->heads_k > BSA_MAX_HEADS)
    return bsa_internal_fail(BSA_ERR_INVALID_ARG, "rope heads_k is out of range");
  const Geo* g = nullptr;
  int is_bf16 = 0, device = -1;
  bsa_status s = bsa_internal_plan_sizes(plan, &g, &is_bf16, &device);
  if (s != BSA_OK) return s;
  if (R < 2 || R > g->D)
    return bsa_internal_fail(BSA_ERR_INVALID_ARG, "rope dims must sum to a number in [2, head_dim]");
  bsa_rope_s* r = new (std::nothrow) bsa_rope_s;
  if (r == nullptr) return bsa_internal_fail(BSA_ERR_CUDA, "out of host memory");
  std::memset(r, 0, sizeof(*r));
  r->g = *g;
  r->is_bf16 = is_bf16;
  r->device = device;
  r->heads_k = c->heads_k ? c->heads_k : g->Hd;
  r->layout = (int)c->layout;
  r->mscale = (float)c->mscale;
  const double two_pi = 6.283185307179586476925;
  int p = 0;
  for (int x = 0; x < 3; ++x) {
    const int d = c->dim[x];
    r->pairs[x] = d / 2;
    double theta = c->theta;
    if (c->scaling == BSA_ROPE_NTK && d > 2) theta *= std::pow(c->factor[x], (double)d / (d - 2));
    for (int i = 0; i < d / 2; ++i) {
      double f = std::pow(theta, -2.0 * i / d);
      if (c->scaling == BSA_ROPE_LINEAR) f /= c->factor[x];
      if (c->scaling == BSA_ROPE_YARN) {
        double keep = (c->orig_len[x] * f / two_pi - c->beta_slow) / (c->beta_fast - c->beta_slow);
        keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
        f = (1.0 - keep) * f / c->factor[x] + keep * f;
      }
      r->turns[p++] = f / two_pi;
    }
  }
  *out = r;
  return BSA_OK;
}

bsa_status bsa_rope_destroy(bsa_rope_t rope) {
  delete rope;
  return BSA_OK;
}

bsa_status bsa_rotary(bsa_rope_t r, const bsa_view_t* q, const bsa_view_t* k, const bsa_view_t* q_out,
                      const bsa_view_t* k_out, const int64_t* t_origin, int backward, void* stream) {
  if (r == nullptr) return bsa_internal_fail(BSA_ERR_INVALID_ARG, "rope is NULL");
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return bsa_internal_fail(BSA_ERR_CUDA, cudaGetErrorString(e));
  if (dev != r->device) return bsa_internal_fail(BSA_ERR_INVALID_ARG, "rope's plan is on another device than the current one");
  if (backward != 0 && backward != 1) return bsa_internal_fail(BSA_ERR_INVALID_ARG, "backward must be 0 or 1");
  if ((k == nullptr) != (k_out == nullptr))
    return bsa_internal_fail(BSA_ERR_INVALID_ARG, "k and k_out must both be given or both be NULL");
  if (reinterpret_cast<uintptr_t>(t_origin) & 7u)
    return bsa_internal_fail(BSA_ERR_INVALID_ARG, "t_origin must be 8-byte aligned");
  const Geo& g = r->g;
  const int esz = r->is_bf16 ? 2 : 4;
  bsa::RotaryArgs a;
  std::memset(&a, 0, sizeof(a));
  a.heads[0] = g.Hd;
  a.heads[1] = r->heads_k;
  const bsa_view_t* in[2] = {q, k};
  const bsa_view_t* out[2] = {q_out, k_out};
  for (int x = 0; x < (k ? 2 : 1); ++x) {
    bsa_status s = bsa::check_view(in[x], x ? "k" : "q", g.B, g.n_tot, a.heads[x], g.D, esz, false, &a.in[x]);
    if (s != BSA_OK) return s;
    s = bsa::check_view(out[x], x ? "k_out" : "q_out", g.B, g.n_tot, a.heads[x], g.D, esz, true, &a.out[x]);
    if (s != BSA_OK) return s;
    a.in_place[x] = bsa::same_view(a.in[x], a.out[x]);
    if (a.in[x].p == a.out[x].p && !a.in_place[x])
      return bsa_internal_fail(BSA_ERR_INVALID_ARG, "an output starts at its input but has other strides");
  }
  if (k && a.out[0].p == a.out[1].p) return bsa_internal_fail(BSA_ERR_INVALID_ARG, "q_out and k_out are the same memory");
  // (threads turn a token's Q before its K, and CTAs in any order)
  if (k && (a.out[0].p == a.in[1].p || a.out[1].p == a.in[0].p))
    return bsa_internal_fail(BSA_ERR_INVALID_ARG, "q_out is the memory of k, or k_out that of q");
  a.rows = (long long)g.B * g.n_tot;
  a.n_video = g.n_video;
  a.div_tot = make_fastdiv((uint32_t)g.n_tot);
  a.div_w = make_fastdiv((uint32_t)g.W);
  a.div_h = make_fastdiv((uint32_t)g.H);
  a.pt = r->pairs[0];
  a.pty = a.pt + r->pairs[1];
  a.pairs = a.pty + r->pairs[2];
  a.mscale = r->mscale;
  a.sine_sign = backward ? -r->mscale : r->mscale;
  a.t_origin = t_origin;
  std::memcpy(a.turns, r->turns, sizeof(a.turns));
  const bool half = r->layout == BSA_ROPE_HALF;
  cudaStream_t st = (cudaStream_t)stream;
  e = r->is_bf16 ? bsa::launch_rotary<__nv_bfloat16>(g, half, a, st) : bsa::launch_rotary<float>(g, half, a, st);
  return e == cudaSuccess ? BSA_OK : bsa_internal_fail(BSA_ERR_CUDA, cudaGetErrorString(e));
}

}  // extern "C"
