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
//
// Measured on the device, in a captured graph (32 query and 8 KV heads of 128): 15k
// prompt tokens into bf16 pages 70 us, 5.5 TB/s on the bytes they need (0.85 of the
// measured copy; as calls, by the wall clock, 72 us and 0.82), into 4 bits with 7.7k
// tokens 51 us, of which the queries take 16, the metadata 9 and the rest
// is bound by issue and by few warps to hide latencies (520 instructions per token and
// KV head, issue slots 62% used); the read-back of 100k tokens 95 us, 5.5 TB/s,
// writes for the most part; one token in each of 64 sequences 5.6 us (4 bits 6.2),
// the chain length, page, keys, metadata.
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
  int heads;  // KV heads (or their query groups) that one CTA takes in turn
};

// The new tokens of one page: slots lo .. hi−1; slot s is row `row + s − lo`.
struct PageItem {
  int phys, lo, hi, row, pos;  // pos: position of slot 0
};

// Called by whole warps; every lane gets the same answer.
template <class A>
__device__ bool page_item(const A& a, int item, PageItem* out) {
  int b = item, row0 = item, n = 1, k = 0, L;
  if (a.indptr != nullptr) {
    // greatest b with base(b) ≤ item, 32 probes at a time: ⌈log32(batch)⌉ rounds, of
    // which the last brings the sequence's rows and length along, then the page
    // table's load (without indptr: the length, then the table)
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = a.batch;
    for (;;) {
      const int step = (hi - lo + 31) >> 5, at = lo + lane * step;
      int first = 0, end = 0, len = 0;
      if (at < hi) {
        first = a.indptr[at];
        if (step == 1) {
          end = a.indptr[at + 1];
          len = a.seq_lens[at];
        }
      }
      const bool le = at < hi && first / a.S + 2 * at <= item;
      const int c = __popc(__ballot_sync(0xffffffffu, le || lane == 0)) - 1;
      lo += c * step;
      if (step == 1) {
        b = lo;
        row0 = __shfl_sync(0xffffffffu, first, c);
        n = __shfl_sync(0xffffffffu, end, c);
        L = __shfl_sync(0xffffffffu, len, c);
        break;
      }
      hi = min(hi, lo + step);
    }
    const int end = n;
    n = end - row0;
    k = item - (row0 / a.S + 2 * b);
    if (row0 < 0 || n < 0 || end > a.rows) {
      raise_flag(EKV_EFLAG_BAD_LEN);
      return false;
    }
  } else {
    L = a.seq_lens[b];
  }
  if (n == 0 || (a.indptr == nullptr && L == 0)) return false;
  if (L < n || L > a.max_pages * a.S) {
    raise_flag(EKV_EFLAG_BAD_LEN);
    return false;
  }
  const int first = L - n, p = first / a.S + k;
  // in 64 bits: behind a sequence that ends near 2^31 lie items whose pages start past it
  if (k < 0 || static_cast<int64_t>(p) * a.S >= L) return false;
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

// A row of d numbers is rotated in units of eight numbers or, for half-split
// pairs, of eight and their eight partners; a unit owns all it reads, so a row
// may be rotated in place.  The threads of a CTA are laid out as a power of two
// of units (slots) by rows, so that nothing is divided.
struct Layout {
  int units, slots;  // units per row, and the power of two above
  int u, r0, step;   // this thread's unit, first row, and the rows of one pass
};
__device__ __forceinline__ Layout row_layout(int D, int rot, int interleaved) {
  Layout l;
  l.units = interleaved ? D / 8 : (D - rot / 2) / 8;
  l.slots = l.units > 8 ? 16 : (l.units > 4 ? 8 : 4);
  const int shift = l.units > 8 ? 4 : (l.units > 4 ? 3 : 2);
  l.u = threadIdx.x & (l.slots - 1);
  l.r0 = threadIdx.x >> shift;
  l.step = kThreads >> shift;
  return l;
}
// Cosines and sines of a unit (as many as it has pairs: eight, four, or none).
struct Turn {
  float c[8], s[8];
};
__device__ __forceinline__ void load_turn(Turn& t, const float* cs, int u, int rot, int interleaved) {
  const int half = rot / 2;
  if (!interleaved && u < half / 8) {
    load8(cs + 8 * u, t.c);
    load8(cs + half + 8 * u, t.s);
  } else if (interleaved && 8 * u < rot) {
    load4(cs + 4 * u, t.c);
    load4(cs + half + 4 * u, t.s);
  }
}
// The raw bits of a unit: its eight numbers, and its partners' where it has any.
template <typename T>
struct Raw {
  uint4 x[sizeof(T) / 2], z[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ void load_raw(Raw<T>& r, const T* src, int u, int rot, int interleaved) {
  const int half = rot / 2;
  const bool split = !interleaved && u < half / 8;
  const T* p = src + (interleaved || split ? 8 * u : half + 8 * u);
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) r.x[i] = reinterpret_cast<const uint4*>(p)[i];
  if (split) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) r.z[i] = reinterpret_cast<const uint4*>(p + half)[i];
  }
}
template <typename T>
__device__ __forceinline__ void widen8(const uint4 (&w)[sizeof(T) / 2], float* v) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t ws[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(ws[i]);
      v[2 * i + 1] = bf16_hi(ws[i]);
    }
  } else {
    const uint32_t ws[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(ws[i]);
  }
}
template <typename T>
__device__ __forceinline__ void rotate_unit(const Raw<T>& r, const Turn& t, T* dst, T* dst2, int u, int rot,
                                            int interleaved) {
  const int half = rot / 2;
  float x[8], y[8];
  widen8<T>(r.x, x);
  if (!interleaved && u < half / 8) {
    float z[8];
    widen8<T>(r.z, z);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = fmaf(x[i], t.c[i], -z[i] * t.s[i]);
      z[i] = fmaf(z[i], t.c[i], x[i] * t.s[i]);
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
  if (interleaved && j < rot) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = fmaf(x[2 * i], t.c[i], -x[2 * i + 1] * t.s[i]);
      y[2 * i + 1] = fmaf(x[2 * i + 1], t.c[i], x[2 * i] * t.s[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i];
  }
  store8(dst + j, y);
  if (dst2) store8(dst2 + j, y);
}

// Rotates the query heads of KV heads h0 .. h1−1 for a page's new tokens: a
// thread keeps its token's angles and takes heads in turn, four rows' loads at
// a time.
template <typename T, int D>
__device__ void rotate_queries(const AppendArgs& a, const PageItem& it, int h0, int h1) {
  const Layout l = row_layout(D, a.rot, a.interleaved);
  const int n = it.hi - it.lo, Hq = a.Hkv * a.G;
  if (l.u >= l.units) return;
  int toks = 1;  // tokens side by side: a power of two, the rest of the rows are heads
  while (toks < n && toks < l.step) toks <<= 1;
  const int tsh = __ffs(toks) - 1, heads = l.step >> tsh;
  const int first = h0 * a.G + (l.r0 >> tsh), last = h1 * a.G;
  for (int t = l.r0 & (toks - 1); t < n; t += toks) {
    Turn turn;
    if (a.rot) load_turn(turn, rotation_row(a, it.pos + it.lo + t), l.u, a.rot, a.interleaved);
    const int row = it.row + t;
    const T* src = static_cast<const T*>(a.q) + row * a.q_stride;
    T* dst = static_cast<T*>(a.q_out) + static_cast<int64_t>(row) * Hq * D;
    constexpr int kAhead = sizeof(T) == 2 ? 4 : 2;
    int hq = first;
    for (; hq + (kAhead - 1) * heads < last; hq += kAhead * heads) {
      Raw<T> raw[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        load_raw<T>(raw[i], src + static_cast<int64_t>(hq + i * heads) * D, l.u, a.rot, a.interleaved);
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        rotate_unit<T>(raw[i], turn, dst + static_cast<int64_t>(hq + i * heads) * D, static_cast<T*>(nullptr), l.u,
                       a.rot, a.interleaved);
    }
    for (; hq < last; hq += heads) {
      Raw<T> raw;
      load_raw<T>(raw, src + static_cast<int64_t>(hq) * D, l.u, a.rot, a.interleaved);
      rotate_unit<T>(raw, turn, dst + static_cast<int64_t>(hq) * D, static_cast<T*>(nullptr), l.u, a.rot,
                     a.interleaved);
    }
  }
}

#define EKV_R4(n) 1.0 / (n), 1.0 / ((n) + 1), 1.0 / ((n) + 2), 1.0 / ((n) + 3)
__constant__ double kReciprocal[33] = {0.0, EKV_R4(1), EKV_R4(5), EKV_R4(9), EKV_R4(13), EKV_R4(17), EKV_R4(21),
                                       EKV_R4(25), EKV_R4(29)};
#undef EKV_R4

// Metadata of one coordinate over tokens 0..n−1 of a page, as meta.cu computes
// it: exact extremes, mean and population variance in float64 in token order
// with one rounding per operation.  P: 16 or 32, at least n; value(t) is called
// for every t < P, in one batch.
template <int P, class F>
__device__ __forceinline__ void column_meta(F value, int n, float* mx, float* mn, double* mean, double* var) {
  float x[P];
#pragma unroll
  for (int t = 0; t < P; ++t) x[t] = value(t);
  float hi = -INFINITY, lo = INFINITY;
  double s = 0.0, v = 0.0;
#pragma unroll
  for (int t = 0; t < P; ++t) {
    if (t < n) {
      hi = fmaxf(hi, x[t]);
      lo = fminf(lo, x[t]);
      s = __dadd_rn(s, static_cast<double>(x[t]));
    }
  }
  // s/n correctly rounded by Markstein's theorem (IBM J. Res. Dev. 34, 1990): with
  // y = 1/n correctly rounded and q = s·y, the rest r = s − q·n is exact and
  // q + r·y rounds to the quotient.  A table of y in place of the division's
  // chain of dependent steps.
  const double dn = static_cast<double>(n), y = kReciprocal[n];
  auto over_n = [&](double a) {
    const double q = __dmul_rn(a, y), r = __fma_rn(-q, dn, a), c = __fma_rn(r, y, q);
    return fabs(a) <= 1.7976931348623157e308 ? c : q;  // infinities and NaN: as they are
  };
  const double m = over_n(s);
#pragma unroll
  for (int t = 0; t < P; ++t) {
    if (t < n) {
      const double d = __dsub_rn(static_cast<double>(x[t]), m);
      v = __dadd_rn(v, __dmul_rn(d, d));
    }
  }
  *mx = hi;
  *mn = lo;
  *mean = m;
  *var = over_n(v);
}

// grid: (items, CTAs for K and V, then as many for the queries); a CTA takes
// a.heads KV heads in turn: the lookup of its page is a chain of dependent loads
// (page_item), which one head of a prompt's page does not pay for.
template <typename T, int D, int S>
__global__ void __launch_bounds__(kThreads, 5) rope_append_kernel(AppendArgs a) {
  grid_dep_enter();
  PageItem it;
  if (!page_item(a, blockIdx.x, &it)) return;
  const int per = (a.Hkv + a.heads - 1) / a.heads;  // CTAs for K and V
  const int y = static_cast<int>(blockIdx.y), h0 = (y < per ? y : y - per) * a.heads, h1 = min(a.Hkv, h0 + a.heads);
  if (y >= per) {
    rotate_queries<T, D>(a, it, h0, h1);
    return;
  }
  __shared__ __align__(16) T tile[S * D];
  const int n = it.hi - it.lo;
  constexpr int kChunk = 16 / sizeof(T), kChunks = D / kChunk, kRows = kThreads / kChunks, kPasses = S / kRows;
  const Layout l = row_layout(D, a.rot, a.interleaved);
  const int vrow = threadIdx.x / kChunks, vcol = (threadIdx.x % kChunks) * kChunk;
  const bool mine = l.u < l.units && l.r0 < n;
  uint4 v[kPasses];
  Raw<T> raw;  // the thread's first row of K
  const T* ksrc = static_cast<const T*>(a.k) + static_cast<int64_t>(it.row) * a.k_stride;
  const T* vsrc = static_cast<const T*>(a.v) + static_cast<int64_t>(it.row) * a.v_stride + vcol;
  auto load = [&](int h) {
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
      v[i] = *reinterpret_cast<const uint4*>(vsrc + min(vrow + i * kRows, n - 1) * a.v_stride + h * D);
    if (mine) load_raw<T>(raw, ksrc + l.r0 * a.k_stride + h * D, l.u, a.rot, a.interleaved);
  };
  load(h0);
  for (int h = h0; h < h1; ++h) {
    const size_t ph = static_cast<size_t>(it.phys) * a.Hkv + h;
    T* kp = static_cast<T*>(a.k_pool) + ph * S * D;
    T* vp = static_cast<T*>(a.v_pool) + ph * S * D;
    // the page's earlier keys, for its metadata: on their way with the new ones
    if (a.box != nullptr)
      for (int i = threadIdx.x; i < it.lo * kChunks; i += kThreads)
        *reinterpret_cast<uint4*>(tile + i * kChunk) = *reinterpret_cast<const uint4*>(kp + i * kChunk);
    if (mine) {
      for (int t = l.r0; t < n; t += l.step) {
        Turn turn;
        const int slot = it.lo + t;
        if (t != l.r0) load_raw<T>(raw, ksrc + t * a.k_stride + h * D, l.u, a.rot, a.interleaved);
        if (a.rot) load_turn(turn, rotation_row(a, it.pos + slot), l.u, a.rot, a.interleaved);
        rotate_unit<T>(raw, turn, kp + slot * D, tile + slot * D, l.u, a.rot, a.interleaved);
      }
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int t = vrow + i * kRows;
      if (t < n) *reinterpret_cast<uint4*>(vp + (it.lo + t) * D + vcol) = v[i];
    }
    if (h + 1 < h1) load(h + 1);  // in flight during this head's metadata
    if (a.box == nullptr) continue;
    __syncthreads();
    const int j = threadIdx.x;
    if (j < D) {
      float mx, mn;
      double mean, var;
      column_meta<S>([&](int t) { return to_f32(tile[t * D + j]); }, it.hi, &mx, &mn, &mean, &var);
      const size_t mh = (static_cast<size_t>(h) * a.num_phys + it.phys) * 2 * D + j;
      T* box = static_cast<T*>(a.box);
      T* mom = static_cast<T*>(a.mom);
      box[mh] = round_store<T>(mx);
      box[mh + D] = round_store<T>(mn);
      mom[mh] = round_store<T>(mean);
      mom[mh + D] = round_store<T>(var);
    }
    if (h + 1 < h1) __syncthreads();  // the tile is read before the next head's keys enter it
  }
}

// A row of numbers, eight to each of W lanes (W a power of two: a warp takes
// 32/W rows at a time), becomes codes.  Nearly every row is decided in fp32 from
// numbers x, each off by at most err (one bound for the row): only where step or
// zero may round to two bf16 numbers, or a quotient is near a border between two
// codes, are the exact numbers asked, exact(e) in 64 bits (rotated keys: 1 row
// and 1 number in some ten thousand).  All in 64 bits cost four times the issue
// slots.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Extremes that a NaN reaches: a row that holds one has no smallest number, and its
// step and zero are NaN.
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ double min_nan(double a, double b) { return b < a || b != b ? b : a; }
__device__ __forceinline__ double max_nan(double a, double b) { return b > a || b != b ? b : a; }
// Step and zero, from the row's extremes: as low halves of two words, whose
// upper halves differ from them where 64 bits have to decide.
struct Pair {
  uint32_t step, zero;
  __device__ __forceinline__ bool unsure() const {
    return step != __byte_perm(step, 0, 0x1010) || zero != __byte_perm(zero, 0, 0x1010) || !(bf16_lo(step) <= 3e38f);
  }
};
__device__ __forceinline__ Pair step_zero(float mn, float mx, float err) {
  // step: off by 2·err/15 of the extremes, and three roundings of fp32
  const float step = (mx - mn) * (1.0f / 15.0f), es = err * 0.14f + step * 0x1p-22f;
  return Pair{bf16_pair(step - es, step + es), bf16_pair(mn - err, mn + err)};
}
template <int W, class F>
__device__ __forceinline__ Pair step_zero_exact(F exact) {
  double mn = exact(0), mx = mn;
#pragma unroll
  for (int e = 1; e < 8; ++e) {
    mn = min_nan(mn, exact(e));
    mx = max_nan(mx, exact(e));
  }
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) {
    mn = min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  // to fp32 and from there to bf16, as the format says
  return Pair{bf16_pair(__double2float_rn((mx - mn) / 15.0), 0.f), bf16_pair(__double2float_rn(mn), 0.f)};
}
// The lane's codes, packed; *packed: the row's (step, zero) as they are stored.  A row
// with a NaN or an infinity gets code 0 and a step that is not finite: NaN as a value.
template <class F>
__device__ __forceinline__ uint32_t row_codes(const float (&x)[8], Pair p, float err, F exact, uint32_t* packed) {
  float step = bf16_lo(p.step);
  const float zero = bf16_lo(p.zero);
  if (step < 1e-30f) step = 0.f;
  // f = (x − zero)/(15·step), clamped to 0 .. 1 as it is formed.  15·f ≤ 15 is off
  // by 15·err·inv, by 2⁻²³ of it for the reciprocal and 2⁻²⁴ for each of 1/15, the
  // product and f (75·2⁻²⁴ < 5e-6), and by 15·2⁻²⁴ of |off| for the rounding of
  // off; adding 1.5·2²³ rounds it to a whole number in the low bits.
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(step));
  inv = step > 0.f ? inv * (1.0f / 15.0f) : 0.f;
  const float off = -zero * inv;
  uint32_t codes = 0;
  float worst = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float f = __saturatef(fmaf(x[e], inv, off)), t = fmaf(f, 15.f, 12582912.f);
    worst = fmaxf(worst, fabsf(fmaf(f, 15.f, 12582912.f - t)));
    codes += __float_as_uint(t) << (4 * e);
  }
  codes -= 0x4b400000u * 0x11111111u;  // eight times the bits of 1.5·2²³
  // (above 2^120 the reciprocal is near the end of its range)
  if (!(worst <= 0.5f - 5e-6f - fabsf(off) * 3e-6f - 15.f * err * inv && step <= 0x1p120f) && step > 0.f) {
    // the code below (a quotient that slips past a whole number changes nothing),
    // and the exact border above it: (n + ½)·step has 13 bits
    codes = 0;
    const double by = static_cast<double>(1.0f / step);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double d = exact(e) - static_cast<double>(zero);
      const float n = floorf(fminf(fmaxf(__double2float_rn(d * by), 0.f), 15.f));
      const double border = static_cast<double>((n + 0.5f) * step);
      const int k = static_cast<int>(n);
      codes |= static_cast<uint32_t>(min(15, k + (d > border || (d == border && (k & 1)) ? 1 : 0))) << (4 * e);
    }
  }
  *packed = (__float_as_uint(step) >> 16) | (__float_as_uint(zero) & 0xffff0000u);
  return codes;
}

// grid as rope_append_kernel; a warp takes the K and V of 256/D tokens at a time,
// eight numbers of each per lane, so that what is worked out once per row is
// shared by two tokens (four of d = 64).  A key's exact rotated numbers, where they
// are asked for: the products are exact in 64 bits (24 + 24 bits), so their sum
// is rounded once, at 2⁻⁵³.
template <typename T, int D, int S>
__global__ void __launch_bounds__(kThreads, 5) rope_append_q4_kernel(AppendArgs a) {
  grid_dep_enter();
  PageItem it;
  if (!page_item(a, blockIdx.x, &it)) return;
  const int per = (a.Hkv + a.heads - 1) / a.heads;  // CTAs for K and V
  const int by = static_cast<int>(blockIdx.y), h0 = (by < per ? by : by - per) * a.heads, h1 = min(a.Hkv, h0 + a.heads);
  if (by >= per) {
    rotate_queries<T, D>(a, it, h0, h1);
    return;
  }
  constexpr int R = q4_record_bytes(D), kRow = D / 2, kLanes = D / 8, kToks = 32 / kLanes, kPass = kThreads / kLanes;
  __shared__ __align__(16) unsigned char codes_s[S * kRow];
  __shared__ uint32_t sz_s[S];
  const int lane = threadIdx.x & 31, in_row = lane % kLanes, n = it.hi - it.lo;
  const int first = static_cast<int>(threadIdx.x) / 32 * kToks, mine = lane / kLanes;  // a warp's first token, the lane's
  const int j = in_row * 8, half = a.rot / 2;
  // this lane's partners and angles: number j + e pairs with j + e + half, − half, or its neighbour
  const bool turns = j < a.rot, low = j < half;
  const int other = !turns || a.interleaved ? j : (low ? j + half : j - half);
  struct Numbers {
    uint4 x[sizeof(T) / 2], z[sizeof(T) / 2], v[sizeof(T) / 2];
  };
  auto load = [&](Numbers& m, int h, int t0) {
    const int64_t row = it.row + min(t0 + mine, n - 1);
    const T* ksrc = static_cast<const T*>(a.k) + row * a.k_stride + h * D;
    const T* vsrc = static_cast<const T*>(a.v) + row * a.v_stride + h * D;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) {
      m.x[i] = reinterpret_cast<const uint4*>(ksrc + j)[i];
      m.z[i] = reinterpret_cast<const uint4*>(ksrc + other)[i];
      m.v[i] = reinterpret_cast<const uint4*>(vsrc + j)[i];
    }
  };
  Numbers next;
  if (first < n) load(next, h0, first);
  for (int h = h0; h < h1; ++h) {
    unsigned char* page = static_cast<unsigned char*>(a.k_pool) +
                          (static_cast<size_t>(it.phys) * a.Hkv + h) * (S / kTile) * R;
    // the page's earlier codes, for its metadata: on their way with the new tokens
    if (a.box != nullptr) {
      for (int i = threadIdx.x; i < it.lo * (kRow / 4); i += kThreads) {
        const int slot = i / (kRow / 4), cc = i - slot * (kRow / 4);
        reinterpret_cast<uint32_t*>(codes_s)[i] =
            reinterpret_cast<const uint32_t*>(page + (slot / kTile) * R + (slot % kTile) * kRow)[cc];
      }
      for (int slot = threadIdx.x; slot < it.lo; slot += kThreads)
        sz_s[slot] = reinterpret_cast<const uint32_t*>(page + (slot / kTile) * R + 16 * D)[slot % kTile];
    }
    for (int t0 = first; t0 < n; t0 += kPass) {
      const int t = min(t0 + mine, n - 1), slot = it.lo + t;
      float c[8], s[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c[e] = 1.f;
        s[e] = 0.f;
      }
      if (turns) {  // number e: x·c − z·s for the first of a pair, x·c + z·s for the second
        const float* cs = rotation_row(a, it.pos + slot);
        if (a.interleaved) {
          float c4[4], s4[4];
          load4(cs + j / 2, c4);
          load4(cs + half + j / 2, s4);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            c[e] = c4[e / 2];
            s[e] = e & 1 ? s4[e / 2] : -s4[e / 2];
          }
        } else {
          const int angle = low ? j : j - half;
          load8(cs + angle, c);
          load8(cs + half + angle, s);
#pragma unroll
          for (int e = 0; e < 8; ++e) s[e] = low ? -s[e] : s[e];
        }
      }
      const Numbers now = next;
      if (t0 + kPass < n) load(next, h, t0 + kPass);  // in flight during this token's work
      else if (h + 1 < h1) load(next, h + 1, first);
      float x[8], z[8], v[8];
      widen8<T>(now.x, x);
      widen8<T>(now.z, z);
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float y = z[e];
          z[e] = z[e + 1];
          z[e + 1] = y;
        }
      }
      widen8<T>(now.v, v);
      // numbers, extremes, and what the rotation's two roundings may be off by
      float y[8], big = 0.f, kmn, kmx, vmn, vmx;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float zs = z[e] * s[e];
        y[e] = fmaf(x[e], c[e], zs);
        big = fmaxf(big, fabsf(y[e]) + fabsf(zs));
        kmn = e ? min_nan(kmn, y[e]) : y[e];
        kmx = e ? max_nan(kmx, y[e]) : y[e];
        vmn = e ? min_nan(vmn, v[e]) : v[e];
        vmx = e ? max_nan(vmx, v[e]) : v[e];
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) {
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
        kmn = min_nan(kmn, __shfl_xor_sync(0xffffffffu, kmn, o));
        kmx = max_nan(kmx, __shfl_xor_sync(0xffffffffu, kmx, o));
        vmn = min_nan(vmn, __shfl_xor_sync(0xffffffffu, vmn, o));
        vmx = max_nan(vmx, __shfl_xor_sync(0xffffffffu, vmx, o));
      }
      const float err = a.rot ? big * 0x1.1p-24f : 0.f;
      auto key = [&](int e) {
        return static_cast<double>(x[e]) * static_cast<double>(c[e]) +
               static_cast<double>(z[e]) * static_cast<double>(s[e]);
      };
      auto value = [&](int e) { return static_cast<double>(v[e]); };
      Pair kp = step_zero(kmn, kmx, err), vp = step_zero(vmn, vmx, 0.f);
      if (__any_sync(0xffffffffu, kp.unsure() || vp.unsure())) {
        kp = step_zero_exact<kLanes>(key);
        vp = step_zero_exact<kLanes>(value);
      }
      uint32_t ksz, vsz;
      const uint32_t kc = row_codes(y, kp, err, key, &ksz), vc = row_codes(v, vp, 0.f, value, &vsz);
      if (t0 + mine >= n) continue;
      unsigned char* rec = page + (slot / kTile) * R;
      const int r = slot % kTile;
      reinterpret_cast<uint32_t*>(rec + r * kRow)[in_row] = kc;
      reinterpret_cast<uint32_t*>(rec + (kTile + r) * kRow)[in_row] = vc;
      reinterpret_cast<uint32_t*>(codes_s + slot * kRow)[in_row] = kc;
      if (in_row == 0) {
        reinterpret_cast<uint32_t*>(rec + 16 * D)[r] = ksz;
        reinterpret_cast<uint32_t*>(rec + 16 * D)[kTile + r] = vsz;
        sz_s[slot] = ksz;
      }
    }
    if (a.box == nullptr) continue;
    __syncthreads();
    const int col = threadIdx.x;
    if (col < D) {
      float mx, mn;
      double mean, var;
      column_meta<S>(
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
    if (h + 1 < h1) __syncthreads();  // the codes are read before the next head's enter
  }
}

struct ReadArgs {
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* indptr;
  const unsigned char* pool;
  void* k_out;
  void* v_out;
  int batch, rows, Hkv, S, num_phys, max_pages;
  int heads;  // KV heads that one CTA takes in turn
};

// grid: (items, CTAs of a.heads KV heads); a thread turns as many codes of K and
// of V into values as 16 bytes hold, so that a warp's stores are one block, two
// tokens of each at a time.  Bound by the values' writes (eight fp32 values per
// thread, in two stores 32 bytes apart, took 240 us for 128k tokens, this 207).
template <typename T>
struct CodesOf {
  using type = uint32_t;
};
template <>
struct CodesOf<float> {
  using type = uint16_t;
};
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) q4_read_kernel(ReadArgs a) {
  grid_dep_enter();
  PageItem it;
  if (!page_item(a, blockIdx.x, &it)) return;
  using Codes = typename CodesOf<T>::type;
  constexpr int E = 16 / sizeof(T), R = q4_record_bytes(D), kWords = D / E, kRows = kThreads / kWords;
  const int w = threadIdx.x % kWords, n = it.hi - it.lo;
  const int h1 = min(a.Hkv, (static_cast<int>(blockIdx.y) + 1) * a.heads);
  // a step: two tokens of one head.  Its codes are loaded while the step before
  // is turned into values.
  struct Step {
    uint32_t codes[2][2], sz[2][2];
  };
  const int first = threadIdx.x / kWords;
  auto load = [&](Step& s, int h, int t0) {
    const unsigned char* page = a.pool + (static_cast<size_t>(it.phys) * a.Hkv + h) * (a.S / kTile) * R;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int slot = it.lo + min(t0 + i * kRows, n - 1);
      const unsigned char* rec = page + (slot / kTile) * R;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const int r = v * kTile + slot % kTile;
        s.codes[i][v] = reinterpret_cast<const Codes*>(rec + r * (D / 2))[w];
        s.sz[i][v] = reinterpret_cast<const uint32_t*>(rec + 16 * D)[r];
      }
    }
  };
  int h = blockIdx.y * a.heads, t0 = first;
  if (t0 >= n) return;
  Step next;
  load(next, h, t0);
  while (h < h1) {
    const Step now = next;
    const int h_now = h, t_now = t0;
    t0 += 2 * kRows;
    if (t0 >= n) {
      t0 = first;
      ++h;
    }
    if (h < h1) load(next, h, t0);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = t_now + i * kRows;
      if (t >= n) continue;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        T* to = static_cast<T*>(v ? a.v_out : a.k_out);
        if (to == nullptr) continue;
        float x[E];
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = q4_value(now.sz[i][v], (now.codes[i][v] >> (4 * e)) & 15u);
        to += (static_cast<int64_t>(it.row + t) * a.Hkv + h_now) * D + E * w;
        if constexpr (E == 8) store8(to, x);
        else *reinterpret_cast<float4*>(to) = make_float4(x[0], x[1], x[2], x[3]);
      }
    }
  }
}

int item_count(const int32_t* indptr, int rows, int batch, int S) {
  return indptr == nullptr ? batch : rows / S + 2 * batch;
}

// KV heads per CTA: about as many as keep the launch to the given waves of five
// CTAs per SM, at least one.  A decode step or a short chunk has one head per
// CTA (latency); in long prompts the page lookups, metadata tails and launches
// of ten times as many CTAs cost more than the waves' ends.  Measured: 15k new
// tokens of 8 KV heads, one head per CTA 84 us, four waves 74.8, two 73.0; the
// read-back of 16k tokens with six waves 19.7, four 16.5, three 15.2, two 15.1, of
// 32k with three 31.2 and two 33.6.
int heads_per_cta(int items, int Hkv, int waves) {
  const int64_t room = 5ll * waves * sm_count();
  const int64_t h = (static_cast<int64_t>(items) * Hkv + room / 2) / (room > 0 ? room : 1);
  return static_cast<int>(h < 1 ? 1 : (h > Hkv ? Hkv : h));
}

template <typename T, int D>
cudaError_t run_append(bool q4, int S, dim3 grid, cudaStream_t st, const AppendArgs& a) {
  if (q4)
    return launch_k(S == 16 ? rope_append_q4_kernel<T, D, 16> : rope_append_q4_kernel<T, D, 32>, grid, kThreads, 0, st, a);
  return launch_k(S == 16 ? rope_append_kernel<T, D, 16> : rope_append_kernel<T, D, 32>, grid, kThreads, 0, st, a);
}

cudaError_t run_append(bool q4, int dtype, int d, const ekv_new_tokens& n, AppendArgs& a, cudaStream_t st) {
  const int items = item_count(n.indptr, n.num_tokens, a.batch, a.S);
  a.heads = heads_per_cta(items, a.Hkv, 2);
  const int per = (a.Hkv + a.heads - 1) / a.heads;
  const dim3 grid(static_cast<unsigned>(items), static_cast<unsigned>(per * (n.q != nullptr ? 2 : 1)));
  if (dtype == EKV_BF16) return d == 128 ? run_append<bf16, 128>(q4, a.S, grid, st, a) : run_append<bf16, 64>(q4, a.S, grid, st, a);
  return d == 128 ? run_append<float, 128>(q4, a.S, grid, st, a) : run_append<float, 64>(q4, a.S, grid, st, a);
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
  return run_append(false, c.dtype, c.head_dim, n, a, st);
}

cudaError_t launch_rope_append_q4(const ekv_cache_q4& c, const ekv_seqs& s, const ekv_rope* rope,
                                  const ekv_new_tokens& n, cudaStream_t st) {
  AppendArgs a = append_args(s, rope, n, c.num_kv_heads, c.page_size, c.num_phys_pages);
  a.k_pool = c.pool;
  a.box = c.box;
  a.mom = c.mom;
  return run_append(true, n.dtype, c.head_dim, n, a, st);
}

cudaError_t launch_q4_read(const ekv_cache_q4& c, const ekv_seqs& s, const int32_t* indptr, int num_tokens,
                           int out_dtype, void* k_out, void* v_out, cudaStream_t st) {
  ReadArgs a{s.page_table, s.seq_lens,     indptr,      static_cast<const unsigned char*>(c.pool),
             k_out,        v_out,          s.batch,     num_tokens,
             c.num_kv_heads, c.page_size,  c.num_phys_pages, s.max_pages, 1};
  const int items = item_count(indptr, num_tokens, s.batch, c.page_size);
  a.heads = heads_per_cta(items, c.num_kv_heads, 3);
  const dim3 grid(static_cast<unsigned>(items), static_cast<unsigned>((c.num_kv_heads + a.heads - 1) / a.heads));
  const bool wide = c.head_dim == 128;
  if (out_dtype == EKV_BF16)
    return launch_k(wide ? q4_read_kernel<bf16, 128> : q4_read_kernel<bf16, 64>, grid, kThreads, 0, st, a);
  return launch_k(wide ? q4_read_kernel<float, 128> : q4_read_kernel<float, 64>, grid, kThreads, 0, st, a);
}

}  // namespace ekv
