// cross_api.cu — the C ABI of cross attention (bsa_cross_*): argument checks,
// the split of each launch, workspace carving and launches.
#include <cfloat>
#include <cmath>
#include <cstring>
#include <new>

#include "bsa.h"
#include "cross.cuh"

bsa_status bsa_internal_tile_map(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims,
                                 const cuuint64_t* strides, const cuuint32_t* box);

struct bsa_cross_s {
  int B, n_q, n_kv, heads, heads_kv, D;
  bsa_dtype dtype;
  int device;
  float scale, scale_log2;
  int32_t* d_status;
  long long wait_limit;      // bound of the tensor-core kernels' waits, SM cycles (0 = default)
  int hold_load;             // test hook of the timeout path (0 = off)
  bsa::CrossTiles fwd, bwd;  // schedules of the forward, and of dQ (and the query tiles of dK, dV) (bf16)
  int fwd_splits, fwd_len;   // partials of a row in the forward, key tiles per split
  int dq_splits, dq_len;     // key splits of dQ
  bool gathers;              // with a key mask, attended K and V rows are copied together first
  int dkv_splits, dkv_len;   // row splits of dK and dV, row tiles in each
};

namespace {

bsa_status fail(bsa_status s, const char* msg) { return bsa_internal_fail(s, msg); }
bsa_status cuda_fail(cudaError_t e) { return fail(BSA_ERR_CUDA, cudaGetErrorString(e)); }
size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

// Splits `units` of work of each of `ctas` CTAs over several CTAs when that
// shortens the call: `slots` CTAs run at a time, each costs about `start` units
// beside its work (its loads before the first product, its stores after the
// last), and a split call about `extra` units more, for writing and merging the
// partials.  Of the splits within `slack` of the least estimate the finest is
// taken that needs no more than four rounds of CTAs.  Returns the units per split, *cost its estimate.
int split_units(long long ctas, long long units, int slots, double start, double extra, double* cost = nullptr,
                double slack = 1.0) {
  long long len = units;
  double best = (double)((ctas + slots - 1) / slots) * (units + start);
  for (int s = 2; s <= 128 && s <= units; ++s) {
    const long long l = (units + s - 1) / s, n = (units + l - 1) / l;
    const double c = (double)((ctas * n + slots - 1) / slots) * (l + start) + extra;
    if (c < best) best = c, len = l;
    else if (c <= slack * best && ctas * n <= 4ll * slots) len = l;
  }
  if (cost) *cost = best;
  return (int)len;
}

constexpr int kSms = 148;

// Query tiles of 128 rows: the divisor of the group that leaves the fewest
// tiles is packed into one (`whole`: only divisors of 128, so that every row of
// a tile is loaded).
void plan_tiles(const bsa_cross_s* c, bool whole, bsa::CrossTiles* t) {
  const int group = c->heads / c->heads_kv;
  long long tiles = 0;
  for (int p = 1; p <= group && p <= 128; ++p) {
    if (group % p || (whole && 128 % p)) continue;
    const int tokens = 128 / p;
    const long long n = (long long)(group / p) * ((c->n_q + tokens - 1) / tokens);
    if (tiles == 0 || n < tiles) tiles = n, t->pack = p, t->tokens = tokens;
  }
  t->tiles = (int)tiles;
  t->bulk_out = 32 % t->pack == 0;
  t->ctas = kSms;
  t->div_hkv = make_fastdiv((uint32_t)c->heads_kv);
  t->div_tok = make_fastdiv((uint32_t)((c->n_q + t->tokens - 1) / t->tokens));
  t->div_pack = make_fastdiv((uint32_t)t->pack);
}

// Items of a K/V head (`per` for each of `splits` key runs).
void plan_items(const bsa_cross_s* c, int per, int splits, bsa::CrossTiles* t) {
  t->items = c->B * c->heads_kv * per * splits;
  t->div_items = make_fastdiv((uint32_t)per);
  t->div_splits = make_fastdiv((uint32_t)splits);
}

// The schedules of the tensor-core kernels.
void plan_tc(bsa_cross_s* c) {
  const long long bh = (long long)c->B * c->heads_kv;
  plan_tiles(c, false, &c->fwd);
  // Two tiles per item over the same keys, or one tile over two runs of keys
  // (always merged): whichever the estimate says ends first, a step of both
  // streams being the unit, an item's start and end about one and a half of them,
  // partials and merge about three.
  const int tiles = c->fwd.tiles;
  c->fwd.step = 128;
  const int steps = (c->n_kv + 127) / 128;
  double pair, dual;
  const int len = split_units(bh * ((tiles + 1) / 2), steps, kSms, 1.5, 3.0, &pair);
  const int half = split_units(bh * tiles, (steps + 1) / 2, kSms, 1.5, 0.0, &dual);
  c->fwd.shared = steps == 1 || pair <= dual + 3.0;
  c->fwd_len = c->fwd.shared ? len : 2 * half;
  const int splits = (steps + c->fwd_len - 1) / c->fwd_len;
  c->fwd_splits = c->fwd.shared ? splits : 2 * splits;
  plan_items(c, c->fwd.shared ? (tiles + 1) / 2 : tiles, splits, &c->fwd);
  const int key_tiles = (c->n_kv + 127) / 128;
  c->bwd.step = 128;
  plan_tiles(c, true, &c->bwd);
  c->bwd.shared = 1;
  const int pairs = (c->bwd.tiles + 1) / 2;
  c->dq_len = split_units(bh * pairs, key_tiles, kSms, 1.0, 2.0);
  c->dq_splits = (key_tiles + c->dq_len - 1) / c->dq_len;
  plan_items(c, pairs, c->dq_splits, &c->bwd);
  // (a CTA whose keys are past its batch element's has nothing to do: finer splits
  // let others take its SM)
  c->dkv_len = split_units(bh * key_tiles, c->bwd.tiles, kSms, 3.0, 2.0, nullptr, 1.07);
  c->dkv_splits = (c->bwd.tiles + c->dkv_len - 1) / c->dkv_len;
}

// The splits of the fp32 kernels: three CTAs of the forward share an SM, two of the
// others.
void plan_f32(bsa_cross_s* c) {
  const long long bh = (long long)c->B * c->heads_kv, rows = (long long)(c->heads / c->heads_kv) * c->n_q;
  const long long row_tiles = (rows + bsa::kCrossF32Rows - 1) / bsa::kCrossF32Rows;
  const long long key_tiles = (c->n_kv + bsa::kCrossF32Keys - 1) / bsa::kCrossF32Keys;
  c->fwd_len = split_units(row_tiles * bh, key_tiles, 3 * kSms, 1.0, 4.0);
  c->fwd_splits = (int)((key_tiles + c->fwd_len - 1) / c->fwd_len);
  c->dq_len = split_units(row_tiles * bh, key_tiles, 2 * kSms, 1.0, 3.0);
  c->dq_splits = (int)((key_tiles + c->dq_len - 1) / c->dq_len);
  const long long kv_rows = (rows + bsa::kCrossF32KvRows - 1) / bsa::kCrossF32KvRows;
  const long long kv_tiles = (c->n_kv + bsa::kCrossF32KvKeys - 1) / bsa::kCrossF32KvKeys;
  c->dkv_len = split_units(kv_tiles * bh, kv_rows, 2 * kSms, 1.0, 3.0);
  c->dkv_splits = (int)((kv_rows + c->dkv_len - 1) / c->dkv_len);
}

// Map (d, head, token, batch) of a [B, n, heads, D] bf16 view with a box of 64
// elements x `pack` heads x `tokens` tokens.  An axis that the view repeats
// (stride 0) becomes one of length 1, its coordinate then stays 0.
bsa_status make_map(CUtensorMap* m, const bsa::View& v, int B, int n, int heads, int D, int pack, int tokens,
                    int* step_b, int* step_h) {
  *step_b = v.b ? 1 : 0;
  *step_h = v.h ? 1 : 0;
  const cuuint64_t any = (cuuint64_t)D * 2;    // stride of an axis of length 1
  const cuuint64_t dims[4] = {(cuuint64_t)D, v.h ? (cuuint64_t)heads : 1, (cuuint64_t)n, v.b ? (cuuint64_t)B : 1};
  const cuuint64_t strides[3] = {v.h ? (cuuint64_t)v.h * 2 : any, v.n ? (cuuint64_t)v.n * 2 : any,
                                 v.b ? (cuuint64_t)v.b * 2 : any};
  const cuuint32_t box[4] = {64, (cuuint32_t)pack, (cuuint32_t)tokens, 1};
  return bsa_internal_tile_map(m, v.p, 4, dims, strides, box);
}

size_t rows_of(const bsa_cross_s* p) { return (size_t)p->B * p->heads * p->n_q; }

size_t counts_bytes(const bsa_cross_s* p) { return round256((size_t)p->B * sizeof(int32_t)); }

// Where a call's workspace begins when it gathers keys: their places, the counts,
// the copies of K and V.
size_t kv_copy_bytes(const bsa_cross_s* p) {
  return round256((size_t)p->B * p->n_kv * p->heads_kv * p->D * (p->dtype == BSA_BF16 ? 2 : 4));
}
size_t gather_bytes(const bsa_cross_s* p) {
  if (!p->gathers) return 0;
  return round256((size_t)p->B * p->n_kv * sizeof(int32_t)) + counts_bytes(p) + 2 * kv_copy_bytes(p);
}

size_t forward_bytes(const bsa_cross_s* p) {
  size_t n = gather_bytes(p);
  if (p->fwd_splits > 1)
    n += round256((size_t)p->fwd_splits * rows_of(p) * p->D * sizeof(float)) +
         round256((size_t)p->fwd_splits * rows_of(p) * sizeof(float2));
  return n;
}

// Backward workspace, after the gathered keys: the row sums (with lse in the query
// tiles' order on the tensor cores), the counts of attended keys, then the partials
// of dQ, whose place those of dK and dV take.
size_t stats_bytes(const bsa_cross_s* p) {
  return p->dtype == BSA_BF16 ? round256((size_t)p->B * p->heads_kv * p->bwd.tiles * 256 * sizeof(float))
                              : round256(rows_of(p) * sizeof(float));
}
size_t backward_bytes(const bsa_cross_s* p) {
  const size_t q = p->dq_splits > 1 ? (size_t)p->dq_splits * rows_of(p) : 0;
  const size_t kv =
      p->dkv_splits > 1 || p->gathers ? (size_t)p->dkv_splits * 2 * p->B * p->heads_kv * p->n_kv : 0;
  return gather_bytes(p) + stats_bytes(p) + counts_bytes(p) + round256((q > kv ? q : kv) * p->D * sizeof(float));
}

// Copies the attended rows of K and V together at the start of `ws` and lets *a
// read them there, without a mask.
cudaError_t gather_keys(const bsa_cross_s* p, char* ws, bsa::CrossArgs* a, cudaStream_t st) {
  a->slot_of = reinterpret_cast<int32_t*>(ws);
  ws += round256((size_t)p->B * p->n_kv * sizeof(int32_t));
  int32_t* counts = reinterpret_cast<int32_t*>(ws);
  ws += counts_bytes(p);
  char *k = ws, *v = ws + kv_copy_bytes(p);
  const cudaError_t e = bsa::launch_cross_gather(*a, counts, k, v, p->D, p->dtype == BSA_BF16, st);
  const long long h = p->heads_kv > 1 ? p->D : 0, n = p->n_kv > 1 ? (long long)p->heads_kv * p->D : 0;
  const long long b = p->B > 1 ? (long long)p->n_kv * p->heads_kv * p->D : 0;
  a->k = bsa::View{k, b, n, h};
  a->v = bsa::View{v, b, n, h};
  a->kv_len = counts;
  a->key_mask = nullptr;
  return e;
}

bsa_status check_cross(const bsa_cross_s* p) {
  if (p == nullptr) return fail(BSA_ERR_INVALID_ARG, "cross is NULL");
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev != p->device) return fail(BSA_ERR_INVALID_ARG, "cross was created on another device than the current one");
  return BSA_OK;
}

bsa_status check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return BSA_OK;
  if (ws == nullptr || have < need) return fail(BSA_ERR_WORKSPACE, "workspace is missing or smaller than bsa_cross_workspace_size says");
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return fail(BSA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  return BSA_OK;
}

// The views and scalars that both directions take.
bsa_status fill(const bsa_cross_s* p, const bsa_view_t* q, const bsa_view_t* k, const bsa_view_t* v,
                const bsa_view_t* o, bool o_written, const float* lse, const int32_t* kv_len,
                const uint8_t* key_mask, int32_t* dev_status, bsa::CrossArgs* a) {
  std::memset(a, 0, sizeof(*a));
  const int esz = p->dtype == BSA_BF16 ? 2 : 4;
  bsa_status s;
  if ((s = bsa::check_view(q, "q", p->B, p->n_q, p->heads, p->D, esz, false, &a->q)) != BSA_OK) return s;
  if ((s = bsa::check_view(k, "k", p->B, p->n_kv, p->heads_kv, p->D, esz, false, &a->k)) != BSA_OK) return s;
  if ((s = bsa::check_view(v, "v", p->B, p->n_kv, p->heads_kv, p->D, esz, false, &a->v)) != BSA_OK) return s;
  if ((s = bsa::check_view(o, "o", p->B, p->n_q, p->heads, p->D, esz, o_written, &a->o)) != BSA_OK) return s;
  if ((p->n_q > 1 && a->q.n == 0) || (p->n_kv > 1 && (a->k.n == 0 || a->v.n == 0)))
    return fail(BSA_ERR_UNSUPPORTED, "cross attention takes no view that repeats its tokens (token stride 0)");
  if (p->heads > 1 && a->q.h == 0)
    return fail(BSA_ERR_UNSUPPORTED, "cross attention takes no query or gradient that repeats its heads (head stride 0)");
  if (reinterpret_cast<uintptr_t>(kv_len) & 3u) return fail(BSA_ERR_INVALID_ARG, "kv_len must be 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(lse) & 3u) return fail(BSA_ERR_INVALID_ARG, "lse must be 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(dev_status) & 3u)
    return fail(BSA_ERR_INVALID_ARG, "dev_status must be 4-byte aligned");
  a->kv_len = kv_len;
  a->key_mask = key_mask;
  a->B = p->B; a->n_q = p->n_q; a->n_kv = p->n_kv; a->heads = p->heads; a->heads_kv = p->heads_kv;
  a->group = p->heads / p->heads_kv;
  a->scale = p->scale;
  a->scale_log2 = p->scale_log2;
  a->status = dev_status ? dev_status : p->d_status;
  return BSA_OK;
}

// The maps of q, k, v (and d_o) for a schedule, whose steps and limits it sets.
bsa_status make_maps(const bsa_cross_s* p, const bsa::CrossArgs& a, bool backward, bsa::CrossMaps* m,
                     bsa::CrossTiles* t) {
  std::memset(m, 0, sizeof(*m));
  bsa_status s;
  if ((s = make_map(&m->q, a.q, p->B, p->n_q, p->heads, p->D, t->pack, t->tokens, &t->step_qb, &t->step_qh)) != BSA_OK ||
      (s = make_map(&m->k, a.k, p->B, p->n_kv, p->heads_kv, p->D, 1, t->step, &t->step_kb, &t->step_kh)) != BSA_OK ||
      (s = make_map(&m->v, a.v, p->B, p->n_kv, p->heads_kv, p->D, 1, t->step, &t->step_vb, &t->step_vh)) != BSA_OK)
    return s;
  if (backward && (s = make_map(&m->d_o, a.d_o, p->B, p->n_q, p->heads, p->D, t->pack, t->tokens, &t->step_ob,
                                &t->step_oh)) != BSA_OK)
    return s;
  int step_b, step_h;      // (an output repeats along no axis)
  if (t->bulk_out && (s = make_map(&m->out, backward ? a.dq : a.o, p->B, p->n_q, p->heads, p->D, t->pack, 32 / t->pack,
                                   &step_b, &step_h)) != BSA_OK)
    return s;
  t->wait_limit = p->wait_limit;
  t->hold_load = p->hold_load;
  return BSA_OK;
}

}  // namespace

extern "C" {

bsa_status bsa_cross_set_watchdog(bsa_cross_t p, long long wait_limit_cycles, int withhold_copy) {
  if (p == nullptr) return fail(BSA_ERR_INVALID_ARG, "cross is NULL");
  if (wait_limit_cycles < 0 || withhold_copy < 0)
    return fail(BSA_ERR_INVALID_ARG, "wait limit and withheld copy must be >= 0");
  p->wait_limit = wait_limit_cycles;
  p->hold_load = withhold_copy;
  return BSA_OK;
}

bsa_status bsa_cross_create(bsa_cross_t* out, int batch, int n_q, int n_kv, int heads, int heads_kv, int head_dim,
                            bsa_dtype dtype, double scale) {
  if (out == nullptr) return fail(BSA_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (batch < 1 || n_q < 1 || n_kv < 1) return fail(BSA_ERR_INVALID_ARG, "batch, n_q and n_kv must be >= 1");
  if (heads < 1 || heads > BSA_MAX_HEADS || heads_kv < 1 || heads % heads_kv)
    return fail(BSA_ERR_INVALID_ARG, "heads must be in [1, 256] and a multiple of heads_kv >= 1");
  if (head_dim != 64 && head_dim != 128) return fail(BSA_ERR_INVALID_ARG, "head_dim must be 64 or 128");
  if (dtype != BSA_F32 && dtype != BSA_BF16) return fail(BSA_ERR_INVALID_ARG, "bad dtype");
  if (!(scale >= 0.0) || !std::isfinite(scale)) return fail(BSA_ERR_INVALID_ARG, "scale must be >= 0");
  if ((long long)batch * heads * (n_q > n_kv ? n_q : n_kv) >= (1ll << 31))
    return fail(BSA_ERR_UNSUPPORTED, "problem exceeds 2^31 rows");
  bsa_cross_s c;
  std::memset(&c, 0, sizeof(c));
  c.B = batch; c.n_q = n_q; c.n_kv = n_kv; c.heads = heads; c.heads_kv = heads_kv; c.D = head_dim;
  c.dtype = dtype;
  const double sc = scale > 0.0 ? scale : 1.0 / std::sqrt((double)head_dim);
  c.scale = (float)sc;
  c.scale_log2 = (float)(sc * 1.4426950408889634);
  if (!(c.scale >= FLT_MIN) || !(c.scale_log2 <= FLT_MAX))
    return fail(BSA_ERR_INVALID_ARG, "scale must be a normal number in fp32");
  if (dtype == BSA_BF16) plan_tc(&c);
  else plan_f32(&c);
  // Gathering costs two launches (8 us together, 1 more per 1024 keys for the scan that
  // numbers them) and a pass over K and V, whatever the mask; how many keys it saves only
  // the device knows.  Forward, gathered against hidden, with 50% / 90% of the keys
  // attended, us: bf16 32 760 queries x 512 keys x 12 heads 80 : 153 / 152 : 124, 2048 x
  // 32 760 x 12 508 : 550 / 535 : 426, 2048 x 2048 x 1 33 : 24 / 33 : 25; fp32 2048 x 1100 x
  // 12 171 : 304 / 279 : 304, 2048 x 32 760 x 1 419 : 631 / 625 : 630, 2048 x 300 x 1 30 : 23 /
  // 31 : 25.  So it pays with many query rows and a mask that hides much, in fp32 at
  // nearly every size, and costs up to 45 us with one K/V head of long keys that are
  // mostly attended.
  c.gathers = (long long)(heads / heads_kv) * n_q >= 2048 && n_kv > 128;
  cudaError_t e = cudaGetDevice(&c.device);
  if (e != cudaSuccess) return cuda_fail(e);
  e = dtype == BSA_F32 ? bsa::prepare_cross_f32(head_dim) : bsa::prepare_cross_tc_forward(c.fwd, head_dim);
  if (e == cudaSuccess && dtype == BSA_BF16) e = bsa::prepare_cross_tc_backward(head_dim);
  if (e == cudaErrorInvalidConfiguration)
    return fail(BSA_ERR_CUDA, "a cross attention kernel was not compiled to the registers per thread that its register "
                              "split assumes (kRegsLaunch): another compiler than the build's");
  if (e == cudaSuccess) e = cudaMalloc(&c.d_status, sizeof(int32_t));
  if (e != cudaSuccess) return cuda_fail(e);
  if ((e = cudaMemset(c.d_status, 0, sizeof(int32_t))) != cudaSuccess ||
      (e = cudaStreamSynchronize(nullptr)) != cudaSuccess) {
    cudaFree(c.d_status);
    return cuda_fail(e);
  }
  *out = new (std::nothrow) bsa_cross_s(c);
  if (*out == nullptr) {
    cudaFree(c.d_status);
    return fail(BSA_ERR_CUDA, "out of host memory");
  }
  return BSA_OK;
}

bsa_status bsa_cross_destroy(bsa_cross_t p) {
  if (p == nullptr) return BSA_OK;
  cudaFree(p->d_status);
  delete p;
  return BSA_OK;
}

bsa_status bsa_cross_workspace_size(bsa_cross_t p, size_t* forward_ws, size_t* backward_ws) {
  if (p == nullptr) return fail(BSA_ERR_INVALID_ARG, "cross is NULL");
  if (forward_ws) *forward_ws = forward_bytes(p);
  if (backward_ws) *backward_ws = backward_bytes(p);
  return BSA_OK;
}

bsa_status bsa_cross_attention(bsa_cross_t p, const bsa_view_t* q, const bsa_view_t* k, const bsa_view_t* v,
                               const int32_t* kv_len, const uint8_t* key_mask, const bsa_view_t* o, float* lse,
                               void* ws, size_t ws_bytes, int32_t* dev_status, void* stream) {
  bsa_status s = check_cross(p);
  if (s != BSA_OK) return s;
  bsa::CrossArgs a;
  if ((s = fill(p, q, k, v, o, true, lse, kv_len, key_mask, dev_status, &a)) != BSA_OK) return s;
  if ((s = check_ws(ws, ws_bytes, forward_bytes(p))) != BSA_OK) return s;
  for (const bsa::View* in : {&a.q, &a.k, &a.v})
    if (a.o.p == in->p) return fail(BSA_ERR_INVALID_ARG, "an output is the memory of an input");
  a.lse = lse;
  a.splits = p->fwd_splits;
  a.split_len = p->fwd_len;
  if (a.splits > 1) {
    char* parts = static_cast<char*>(ws) + gather_bytes(p);
    a.part_o = reinterpret_cast<float*>(parts);
    a.part_ml = reinterpret_cast<float2*>(parts + round256((size_t)a.splits * rows_of(p) * p->D * sizeof(float)));
  }
  cudaStream_t st = (cudaStream_t)stream;
  const bool is_bf16 = p->dtype == BSA_BF16;
  cudaError_t e = cudaSuccess;
  if (p->gathers && key_mask && (e = gather_keys(p, static_cast<char*>(ws), &a, st)) != cudaSuccess) return cuda_fail(e);
  if (is_bf16) {
    bsa::CrossMaps maps;
    bsa::CrossTiles t = p->fwd;
    if ((s = make_maps(p, a, false, &maps, &t)) != BSA_OK) return s;
    e = bsa::launch_cross_tc_forward(a, t, maps, p->D, st);
  } else {
    e = bsa::launch_cross_f32_forward(a, p->D, st);
  }
  if (e == cudaSuccess && a.splits > 1) e = bsa::launch_cross_merge(a, p->D, is_bf16, st);
  return e == cudaSuccess ? BSA_OK : cuda_fail(e);
}

bsa_status bsa_cross_attention_backward(bsa_cross_t p, const bsa_view_t* q, const bsa_view_t* k, const bsa_view_t* v,
                                        const int32_t* kv_len, const uint8_t* key_mask, const bsa_view_t* o,
                                        const float* lse, const bsa_view_t* d_o, const bsa_view_t* dq,
                                        const bsa_view_t* dk, const bsa_view_t* dv, void* ws, size_t ws_bytes,
                                        int32_t* dev_status, void* stream) {
  bsa_status s = check_cross(p);
  if (s != BSA_OK) return s;
  bsa::CrossArgs a;
  if ((s = fill(p, q, k, v, o, false, lse, kv_len, key_mask, dev_status, &a)) != BSA_OK) return s;
  const int esz = p->dtype == BSA_BF16 ? 2 : 4;
  if ((s = bsa::check_view(d_o, "d_o", p->B, p->n_q, p->heads, p->D, esz, false, &a.d_o)) != BSA_OK) return s;
  if ((s = bsa::check_view(dq, "dq", p->B, p->n_q, p->heads, p->D, esz, true, &a.dq)) != BSA_OK) return s;
  if ((s = bsa::check_view(dk, "dk", p->B, p->n_kv, p->heads_kv, p->D, esz, true, &a.dk)) != BSA_OK) return s;
  if ((s = bsa::check_view(dv, "dv", p->B, p->n_kv, p->heads_kv, p->D, esz, true, &a.dv)) != BSA_OK) return s;
  if (lse == nullptr) return fail(BSA_ERR_INVALID_ARG, "lse is NULL");
  if (a.dq.p == a.dk.p || a.dq.p == a.dv.p || a.dk.p == a.dv.p)
    return fail(BSA_ERR_INVALID_ARG, "dq, dk and dv are the same memory");
  for (const bsa::View* out : {&a.dq, &a.dk, &a.dv})
    for (const bsa::View* in : {&a.q, &a.k, &a.v, &a.o, &a.d_o})
      if (out->p == in->p) return fail(BSA_ERR_INVALID_ARG, "an output is the memory of an input");
  if ((s = check_ws(ws, ws_bytes, backward_bytes(p))) != BSA_OK) return s;
  if (p->n_q > 1 && a.d_o.n == 0)
    return fail(BSA_ERR_UNSUPPORTED, "cross attention takes no view that repeats its tokens (token stride 0)");
  if (p->heads > 1 && a.d_o.h == 0)
    return fail(BSA_ERR_UNSUPPORTED, "cross attention takes no query or gradient that repeats its heads (head stride 0)");
  const bool is_bf16 = p->dtype == BSA_BF16;
  a.lse = const_cast<float*>(lse);
  char* sums = static_cast<char*>(ws) + gather_bytes(p);
  a.delta = a.stats = reinterpret_cast<float*>(sums);
  a.part_o = a.part_kv = reinterpret_cast<float*>(sums + stats_bytes(p) + counts_bytes(p));
  if (key_mask && !p->gathers) a.attended = reinterpret_cast<int32_t*>(sums + stats_bytes(p));
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  if (p->gathers && key_mask && (e = gather_keys(p, static_cast<char*>(ws), &a, st)) != cudaSuccess) return cuda_fail(e);
  bsa::CrossMaps maps;
  bsa::CrossTiles t = p->bwd;
  if (is_bf16 && (s = make_maps(p, a, true, &maps, &t)) != BSA_OK) return s;
  e = is_bf16 ? bsa::launch_cross_stats(a, t, p->D, st) : bsa::launch_cross_delta(a, p->D, st);
  a.splits = p->dq_splits;
  a.split_len = p->dq_len;
  if (e == cudaSuccess)
    e = is_bf16 ? bsa::launch_cross_tc_dq(a, t, maps, p->D, st) : bsa::launch_cross_f32_dq(a, p->D, st);
  if (e == cudaSuccess && a.splits > 1) e = bsa::launch_cross_sum_q(a, p->D, is_bf16, st);
  a.splits = p->dkv_splits;
  a.split_len = p->dkv_len;
  if (e == cudaSuccess)
    e = is_bf16 ? bsa::launch_cross_tc_dkv(a, t, maps, p->D, st) : bsa::launch_cross_f32_dkv(a, p->D, st);
  if (e == cudaSuccess && (a.splits > 1 || a.slot_of)) e = bsa::launch_cross_reduce_kv(a, p->D, is_bf16, st);
  return e == cudaSuccess ? BSA_OK : cuda_fail(e);
}

bsa_status bsa_cross_check_status(bsa_cross_t p, void* stream) {
  bsa_status s = check_cross(p);
  if (s != BSA_OK) return s;
  cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
  int32_t v = 0;
  if (e == cudaSuccess) e = cudaMemcpy(&v, p->d_status, sizeof(v), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemset(p->d_status, 0, sizeof(v));
  if (e != cudaSuccess) return cuda_fail(e);
  if (v == 0) return BSA_OK;
  return fail((bsa_status)v, v == BSA_ERR_TIMEOUT ? "kernel reported that a bounded wait ran out"
                                                   : "kernel reported a kv_len outside [0, n_kv]");
}

}  // extern "C"
