// The cache append with the position rotation applied on the way, into a bf16
// or fp32 paged cache and into a 4-bit one, and the read-back of the latter
// (include/ekv.h: ekv_rope_append, ekv_rope_append_q4, ekv_q4_read).
//
// One CTA owns one (page, KV head) that received tokens: it rotates its keys,
// writes K and V, and refreshes the page's metadata (EntmaxKV summary page,
// gist.science/fr/paper/2605.21649, §2.A) from the tile it holds in shared
// memory, so a prompt's K is read once and no second pass builds its metadata.
// Further CTAs rotate the query heads of the same page's tokens.  A page has
// one owner, so nothing is written twice and no result depends on an order.
//
// Which pages a ragged batch touches is known on the device only.  Item i
// maps to sequence b by base(b) = ⌊indptr[b]/S⌋ + 2b: n new tokens touch at most
// ⌊n/S⌋ + 2 pages and base(b+1) − base(b) ≥ ⌊n/S⌋ + 2, so the items of a
// sequence never reach the next one's, and ⌊rows/S⌋ + 2·batch items are enough
// without a prefix sum over the batch.
#include "q4.cuh"

namespace ekv {

namespace {

constexpr int kThreads = 128;

struct AppendArgs {
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* indptr;
  const float* cos_sin;
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  void* k_pool;  // the 4-bit pool, for a 4-bit cache
  void* v_pool;
  void* box;
  void* mom;
  int64_t q_stride, k_stride, v_stride;
  int max_pos, rot, interleaved;
  int batch, rows, Hkv, G, S, num_phys, max_pages;
};

// The new tokens of one page: slots lo .. hi−1; slot s is row `row + s − lo`.
struct PageItem {
  int phys, lo, hi, row, pos;  // pos: position of slot 0
};

// Called by whole warps; every lane gets the same answer.
template <class A>
__device__ bool page_item(const A& a, int item, PageItem* out) {
  int b = item, row0 = item, n = 1, k = 0;
  if (a.indptr != nullptr) {
    // greatest b with base(b) ≤ item, 32 probes at a time
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = a.batch;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) >> 5;
      const int at = lo + lane * step;
      const bool le = at < hi && a.indptr[at] / a.S + 2 * at <= item;
      const int c = __popc(__ballot_sync(0xffffffffu, le || lane == 0));
      lo += (c - 1) * step;
      hi = min(hi, lo + step);
    }
    b = lo;
    row0 = a.indptr[b];
    const int end = a.indptr[b + 1];
    n = end - row0;
    k = item - (row0 / a.S + 2 * b);
    if (row0 < 0 || n < 0 || end > a.rows) {
      raise_flag(EKV_EFLAG_BAD_LEN);
      return false;
    }
  }
  const int L = a.seq_lens[b];
  if (n == 0 || (a.indptr == nullptr && L == 0)) return false;
  if (L < n || L > a.max_pages * a.S) {
    raise_flag(EKV_EFLAG_BAD_LEN);
    return false;
  }
  const int first = L - n, p = first / a.S + k;
  if (k < 0 || p * a.S >= L) return false;
  const int phys = a.page_table[static_cast<size_t>(b) * a.max_pages + p];
  if (!phys_ok(phys, a.num_phys)) return false;
  out->phys = phys;
  out->lo = max(0, first - p * a.S);
  out->hi = min(a.S, L - p * a.S);
  out->pos = p * a.S;
  out->row = row0 + p * a.S + out->lo - first;
  return true;
}

__device__ __forceinline__ const float* rotation_row(const AppendArgs& a, int pos) {
  if (pos >= a.max_pos) {
    raise_flag(EKV_EFLAG_BAD_POS);
    pos = a.max_pos - 1;
  }
  return a.cos_sin + static_cast<size_t>(pos) * a.rot;
}

__device__ __forceinline__ void store8(bf16* p, const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&r);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// Units of work of one row of d numbers, eight or twice eight of them each:
// half-split pairs take chunk u of the first half of rot with its partner;
// everything else is one chunk.  A unit owns all it reads, so a row may be
// rotated in place.
__device__ __forceinline__ int row_units(int D, int rot, int interleaved) {
  return interleaved ? D / 8 : (D - rot / 2) / 8;
}
template <typename T>
__device__ __forceinline__ void rotate_unit(const T* src, T* dst, T* dst2, const float* cs, int u, int rot,
                                            int interleaved) {
  const int half = rot / 2;
  float x[8], y[8];
  if (!interleaved && u < half / 8) {
    float z[8], c[8], s[8];
    load8(src + 8 * u, x);
    load8(src + half + 8 * u, z);
    load8(cs + 8 * u, c);
    load8(cs + half + 8 * u, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = fmaf(x[i], c[i], -z[i] * s[i]);
      z[i] = fmaf(z[i], c[i], x[i] * s[i]);
    }
    store8(dst + 8 * u, y);
    store8(dst + half + 8 * u, z);
    if (dst2) {
      store8(dst2 + 8 * u, y);
      store8(dst2 + half + 8 * u, z);
    }
    return;
  }
  const int j = interleaved ? 8 * u : half + 8 * u;
  load8(src + j, x);
  if (interleaved && j < rot) {
    float c[4], s[4];
    load4(cs + j / 2, c);
    load4(cs + half + j / 2, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = fmaf(x[2 * i], c[i], -x[2 * i + 1] * s[i]);
      y[2 * i + 1] = fmaf(x[2 * i + 1], c[i], x[2 * i] * s[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i];
  }
  store8(dst + j, y);
  if (dst2) store8(dst2 + j, y);
}

// Rotates the G query heads of KV head h for a page's new tokens.
template <typename T, int D>
__device__ void rotate_queries(const AppendArgs& a, const PageItem& it, int h) {
  const int units = row_units(D, a.rot, a.interleaved), per_tok = units * a.G, n = it.hi - it.lo;
  const int Hq = a.Hkv * a.G;
  for (int i = threadIdx.x; i < n * per_tok; i += kThreads) {
    const int t = i / per_tok, r = i - t * per_tok, g = r / units, u = r - g * units;
    const int row = it.row + t, head = h * a.G + g;
    const float* cs = a.rot ? rotation_row(a, it.pos + it.lo + t) : nullptr;
    rotate_unit<T>(static_cast<const T*>(a.q) + row * a.q_stride + static_cast<int64_t>(head) * D,
                   static_cast<T*>(a.q_out) + (static_cast<int64_t>(row) * Hq + head) * D, nullptr, cs, u, a.rot,
                   a.interleaved);
  }
}

// Metadata of one coordinate over tokens 0..n−1 of a page, as meta.cu computes
// it: exact extremes, mean and population variance in float64 in token order
// with one rounding per operation.
template <class F>
__device__ __forceinline__ void column_meta(F value, int n, float* mx, float* mn, double* mean, double* var) {
  float hi = -INFINITY, lo = INFINITY;
  double s = 0.0, v = 0.0;
  for (int t = 0; t < n; ++t) {
    const float x = value(t);
    hi = fmaxf(hi, x);
    lo = fminf(lo, x);
    s = __dadd_rn(s, static_cast<double>(x));
  }
  const double dn = static_cast<double>(n), m = __ddiv_rn(s, dn);
  for (int t = 0; t < n; ++t) {
    const double d = __dsub_rn(static_cast<double>(value(t)), m);
    v = __dadd_rn(v, __dmul_rn(d, d));
  }
  *mx = hi;
  *mn = lo;
  *mean = m;
  *var = __ddiv_rn(v, dn);
}

// grid: (items, Hkv for K and V, then Hkv more for the queries).
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(AppendArgs a) {
  grid_dep_enter();
  PageItem it;
  if (!page_item(a, blockIdx.x, &it)) return;
  if (static_cast<int>(blockIdx.y) >= a.Hkv) {
    rotate_queries<T, D>(a, it, blockIdx.y - a.Hkv);
    return;
  }
  __shared__ __align__(16) T tile[32 * D];
  const int h = blockIdx.y, n = it.hi - it.lo;
  const size_t ph = static_cast<size_t>(it.phys) * a.Hkv + h;
  T* kp = static_cast<T*>(a.k_pool) + ph * a.S * D;
  T* vp = static_cast<T*>(a.v_pool) + ph * a.S * D;
  constexpr int kChunk = 16 / sizeof(T), kChunks = D / kChunk;
  const T* vsrc = static_cast<const T*>(a.v) + static_cast<int64_t>(h) * D;
  for (int i = threadIdx.x; i < n * kChunks; i += kThreads) {
    const int t = i / kChunks, c = (i - t * kChunks) * kChunk;
    *reinterpret_cast<uint4*>(vp + (it.lo + t) * D + c) =
        *reinterpret_cast<const uint4*>(vsrc + (it.row + t) * a.v_stride + c);
  }
  const int units = row_units(D, a.rot, a.interleaved);
  const T* ksrc = static_cast<const T*>(a.k) + static_cast<int64_t>(h) * D;
  for (int i = threadIdx.x; i < n * units; i += kThreads) {
    const int t = i / units, u = i - t * units, slot = it.lo + t;
    const float* cs = a.rot ? rotation_row(a, it.pos + slot) : nullptr;
    rotate_unit<T>(ksrc + (it.row + t) * a.k_stride, kp + slot * D, tile + slot * D, cs, u, a.rot, a.interleaved);
  }
  if (a.box == nullptr) return;
  for (int i = threadIdx.x; i < it.lo * kChunks; i += kThreads)
    *reinterpret_cast<uint4*>(tile + i * kChunk) = *reinterpret_cast<const uint4*>(kp + i * kChunk);
  __syncthreads();
  const int j = threadIdx.x;
  if (j >= D) return;
  float mx, mn;
  double mean, var;
  column_meta([&](int t) { return to_f32(tile[t * D + j]); }, it.hi, &mx, &mn, &mean, &var);
  const size_t mh = (static_cast<size_t>(h) * a.num_phys + it.phys) * 2 * D + j;
  T* box = static_cast<T*>(a.box);
  T* mom = static_cast<T*>(a.mom);
  box[mh] = round_store<T>(mx);
  box[mh + D] = round_store<T>(mn);
  mom[mh] = round_store<T>(mean);
  mom[mh + D] = round_store<T>(var);
}

// One row of D numbers, D/32 of them per lane (in 64 bits), to codes: the
// lane's codes come back packed, the pair (step, zero) on every lane.  The
// quotient runs in fp32, off by at most 3·2⁻²⁴·15.5 < 3e-6; within 2e-5 of a
// border between two codes it is divided again in 64 bits.
template <int E>
__device__ __forceinline__ uint32_t quantise_row(const double (&y)[E], uint32_t* step_zero) {
  double mn = y[0], mx = y[0];
#pragma unroll
  for (int e = 1; e < E; ++e) {
    mn = fmin(mn, y[e]);
    mx = fmax(mx, y[e]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mn = fmin(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = fmax(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  bf16 sb = __float2bfloat16_rn(__double2float_rn((mx - mn) / 15.0));
  if (!(__bfloat162float(sb) >= 1e-30f)) sb = __ushort_as_bfloat16(0);
  const bf16 zb = __float2bfloat16_rn(__double2float_rn(mn));
  const float step = __bfloat162float(sb), inv = step > 0.f ? 1.0f / step : 0.f;
  const double zero = __bfloat162float(zb);
  uint32_t codes = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const double d = y[e] - zero;
    const float f = __double2float_rn(d) * inv;
    float n = rintf(f);
    if (fabsf(f - n) > 0.5f - 2e-5f && step > 0.f) n = __double2float_rn(rint(d / static_cast<double>(step)));
    codes |= static_cast<uint32_t>(fminf(fmaxf(n, 0.f), 15.f)) << (4 * e);
  }
  *step_zero = static_cast<uint32_t>(__bfloat16_as_ushort(sb)) |
               (static_cast<uint32_t>(__bfloat16_as_ushort(zb)) << 16);
  return codes;
}

template <typename T, int E>
__device__ __forceinline__ void load_lane(const T* p, float (&v)[E]) {
  if constexpr (E == 4) {
    load4(p, v);
  } else if constexpr (sizeof(T) == 2) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
    v[0] = bf16_lo(w);
    v[1] = bf16_hi(w);
  } else {
    const float2 w = *reinterpret_cast<const float2*>(p);
    v[0] = w.x;
    v[1] = w.y;
  }
}

// grid as rope_append_kernel; a warp takes one row (K or V of one token) at a
// time, D/32 numbers per lane.  The products of the rotation are exact in 64
// bits (24 + 24 bits), so its sums are rounded once, at 2⁻⁵³.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) rope_append_q4_kernel(AppendArgs a) {
  grid_dep_enter();
  PageItem it;
  if (!page_item(a, blockIdx.x, &it)) return;
  if (static_cast<int>(blockIdx.y) >= a.Hkv) {
    rotate_queries<T, D>(a, it, blockIdx.y - a.Hkv);
    return;
  }
  constexpr int E = D / 32, R = q4_record_bytes(D), kRow = D / 2;
  __shared__ __align__(16) unsigned char codes_s[32 * kRow];
  __shared__ uint32_t sz_s[32];
  const int h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = it.hi - it.lo;
  unsigned char* page = static_cast<unsigned char*>(a.k_pool) +
                        (static_cast<size_t>(it.phys) * a.Hkv + h) * (a.S / kTile) * R;
  const int j = lane * E, half = a.rot / 2;
  for (int i = warp; i < 2 * n; i += kThreads / 32) {
    const int t = i >> 1, isv = i & 1, slot = it.lo + t;
    double y[E];
    float x[E];
    if (isv) {
      load_lane<T, E>(static_cast<const T*>(a.v) + (it.row + t) * a.v_stride + h * D + j, x);
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = x[e];
    } else {
      const T* src = static_cast<const T*>(a.k) + (it.row + t) * a.k_stride + h * D;
      load_lane<T, E>(src + j, x);
      if (j < a.rot) {
        const float* cs = rotation_row(a, it.pos + slot);
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const double c = cs[(j + e) / 2], s = cs[half + (j + e) / 2];
            y[e] = static_cast<double>(x[e]) * c - static_cast<double>(x[e + 1]) * s;
            y[e + 1] = static_cast<double>(x[e + 1]) * c + static_cast<double>(x[e]) * s;
          }
        } else {
          const bool low = j < half;
          const int jj = low ? j : j - half;
          float z[E], c[E], s[E];
          load_lane<T, E>(src + (low ? j + half : jj), z);
          load_lane<float, E>(cs + jj, c);
          load_lane<float, E>(cs + half + jj, s);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const double zs = static_cast<double>(z[e]) * static_cast<double>(s[e]);
            y[e] = static_cast<double>(x[e]) * static_cast<double>(c[e]) + (low ? -zs : zs);
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = x[e];
      }
    }
    uint32_t sz;
    const uint32_t codes = quantise_row<E>(y, &sz);
    unsigned char* rec = page + (slot / kTile) * R;
    const int r = slot % kTile;
    unsigned char* to = rec + (isv * kTile + r) * kRow;
    if constexpr (E == 4) {
      reinterpret_cast<uint16_t*>(to)[lane] = static_cast<uint16_t>(codes);
      if (!isv) reinterpret_cast<uint16_t*>(codes_s + slot * kRow)[lane] = static_cast<uint16_t>(codes);
    } else {
      to[lane] = static_cast<unsigned char>(codes);
      if (!isv) codes_s[slot * kRow + lane] = static_cast<unsigned char>(codes);
    }
    if (lane == 0) {
      reinterpret_cast<uint32_t*>(rec + 16 * D)[isv * kTile + r] = sz;
      if (!isv) sz_s[slot] = sz;
    }
  }
  if (a.box == nullptr) return;
  for (int i = threadIdx.x; i < it.lo * (kRow / 4); i += kThreads) {
    const int slot = i / (kRow / 4), c = i - slot * (kRow / 4);
    reinterpret_cast<uint32_t*>(codes_s)[i] =
        reinterpret_cast<const uint32_t*>(page + (slot / kTile) * R + (slot % kTile) * kRow)[c];
  }
  for (int slot = threadIdx.x; slot < it.lo; slot += kThreads)
    sz_s[slot] = reinterpret_cast<const uint32_t*>(page + (slot / kTile) * R + 16 * D)[slot % kTile];
  __syncthreads();
  const int col = threadIdx.x;
  if (col >= D) return;
  float mx, mn;
  double mean, var;
  column_meta(
      [&](int t) { return q4_value(sz_s[t], (codes_s[t * kRow + col / 2] >> (4 * (col & 1))) & 15u); }, it.hi, &mx,
      &mn, &mean, &var);
  const size_t mh = (static_cast<size_t>(h) * a.num_phys + it.phys) * 2 * D + col;
  bf16* box = static_cast<bf16*>(a.box);
  bf16* mom = static_cast<bf16*>(a.mom);
  box[mh] = bf16_away(mx, true);
  box[mh + D] = bf16_away(mn, false);
  mom[mh] = round_store<bf16>(mean);
  mom[mh + D] = round_store<bf16>(var);
}

struct ReadArgs {
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* indptr;
  const unsigned char* pool;
  void* k_out;
  void* v_out;
  int batch, rows, Hkv, S, num_phys, max_pages;
};

// grid: (items, Hkv); a thread turns eight codes (one word) into values.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) q4_read_kernel(ReadArgs a) {
  grid_dep_enter();
  PageItem it;
  if (!page_item(a, blockIdx.x, &it)) return;
  constexpr int R = q4_record_bytes(D), kWords = D / 8;
  const int h = blockIdx.y, n = it.hi - it.lo;
  const unsigned char* page = a.pool + (static_cast<size_t>(it.phys) * a.Hkv + h) * (a.S / kTile) * R;
  for (int i = threadIdx.x; i < 2 * n * kWords; i += kThreads) {
    const int row = i / kWords, w = i - row * kWords, isv = row >= n, t = isv ? row - n : row, slot = it.lo + t;
    T* to = static_cast<T*>(isv ? a.v_out : a.k_out);
    if (to == nullptr) continue;
    const unsigned char* rec = page + (slot / kTile) * R;
    const int r = isv * kTile + slot % kTile;
    const uint32_t codes = reinterpret_cast<const uint32_t*>(rec + r * (D / 2))[w];
    const uint32_t sz = reinterpret_cast<const uint32_t*>(rec + 16 * D)[r];
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = q4_value(sz, (codes >> (4 * e)) & 15u);
    store8(to + (static_cast<int64_t>(it.row + t) * a.Hkv + h) * D + 8 * w, v);
  }
}

int item_count(const int32_t* indptr, int rows, int batch, int S) {
  return indptr == nullptr ? batch : rows / S + 2 * batch;
}

AppendArgs append_args(const ekv_seqs& s, const ekv_rope* rope, const ekv_new_tokens& n, int Hkv, int S,
                       int num_phys) {
  AppendArgs a{};
  a.page_table = s.page_table;
  a.seq_lens = s.seq_lens;
  a.indptr = n.indptr;
  if (rope != nullptr) {
    a.cos_sin = rope->cos_sin;
    a.max_pos = rope->max_pos;
    a.rot = rope->rot_dim;
    a.interleaved = rope->interleaved != 0;
  }
  a.q = n.q;
  a.k = n.k;
  a.v = n.v;
  a.q_out = n.q_out;
  a.q_stride = n.q_stride;
  a.k_stride = n.k_stride;
  a.v_stride = n.v_stride;
  a.batch = s.batch;
  a.rows = n.num_tokens;
  a.Hkv = Hkv;
  a.G = n.q != nullptr ? n.num_q_heads / Hkv : 0;
  a.S = S;
  a.num_phys = num_phys;
  a.max_pages = s.max_pages;
  return a;
}

}  // namespace

cudaError_t launch_rope_append(const ekv_cache& c, const ekv_seqs& s, const ekv_rope* rope,
                               const ekv_new_tokens& n, cudaStream_t st) {
  AppendArgs a = append_args(s, rope, n, c.num_kv_heads, c.page_size, c.num_phys_pages);
  a.k_pool = c.k_pool;
  a.v_pool = c.v_pool;
  a.box = c.box;
  a.mom = c.mom;
  const int items = item_count(n.indptr, n.num_tokens, s.batch, c.page_size);
  const dim3 grid(static_cast<unsigned>(items), static_cast<unsigned>(a.Hkv * (n.q != nullptr ? 2 : 1)));
  const bool wide = c.head_dim == 128;
  if (c.dtype == EKV_BF16)
    return launch_k(wide ? rope_append_kernel<bf16, 128> : rope_append_kernel<bf16, 64>, grid, kThreads, 0, st, a);
  return launch_k(wide ? rope_append_kernel<float, 128> : rope_append_kernel<float, 64>, grid, kThreads, 0, st, a);
}

cudaError_t launch_rope_append_q4(const ekv_cache_q4& c, const ekv_seqs& s, const ekv_rope* rope,
                                  const ekv_new_tokens& n, cudaStream_t st) {
  AppendArgs a = append_args(s, rope, n, c.num_kv_heads, c.page_size, c.num_phys_pages);
  a.k_pool = c.pool;
  a.box = c.box;
  a.mom = c.mom;
  const int items = item_count(n.indptr, n.num_tokens, s.batch, c.page_size);
  const dim3 grid(static_cast<unsigned>(items), static_cast<unsigned>(a.Hkv * (n.q != nullptr ? 2 : 1)));
  const bool wide = c.head_dim == 128;
  if (n.dtype == EKV_BF16)
    return launch_k(wide ? rope_append_q4_kernel<bf16, 128> : rope_append_q4_kernel<bf16, 64>, grid, kThreads, 0, st,
                    a);
  return launch_k(wide ? rope_append_q4_kernel<float, 128> : rope_append_q4_kernel<float, 64>, grid, kThreads, 0, st,
                  a);
}

cudaError_t launch_q4_read(const ekv_cache_q4& c, const ekv_seqs& s, const int32_t* indptr, int num_tokens,
                           int out_dtype, void* k_out, void* v_out, cudaStream_t st) {
  ReadArgs a{s.page_table, s.seq_lens,     indptr,      static_cast<const unsigned char*>(c.pool),
             k_out,        v_out,          s.batch,     num_tokens,
             c.num_kv_heads, c.page_size,  c.num_phys_pages, s.max_pages};
  const dim3 grid(static_cast<unsigned>(item_count(indptr, num_tokens, s.batch, c.page_size)),
                  static_cast<unsigned>(c.num_kv_heads));
  const bool wide = c.head_dim == 128;
  if (out_dtype == EKV_BF16)
    return launch_k(wide ? q4_read_kernel<bf16, 128> : q4_read_kernel<bf16, 64>, grid, kThreads, 0, st, a);
  return launch_k(wide ? q4_read_kernel<float, 128> : q4_read_kernel<float, 64>, grid, kThreads, 0, st, a);
}

}  // namespace ekv
