// Softmax decode with capped, biased and masked scores over a paged cache held
// in bf16 or in 4 bits (include/ekv.h: ekv_softmax_decode_mod,
// ekv_softmax_decode_q4), for the G query heads of a KV head times T query
// tokens, at most 64 query rows.
//
// The work is a list of 16-token tiles: those with a visible token, or those
// of the selected pages, of every (sequence, KV head) in turn.  One wave of
// CTAs cuts the whole list into equal runs, whatever the lengths of a ragged
// batch, so every SM streams the same number of bytes; a CTA walks its run
// unit by unit.  Within a unit its warps take every NS-th tile through a
// private ring of bulk copies and keep an online softmax each (running
// maximum, sum, p·v); at the unit's end they are added in warp order.  A unit
// cut by a CTA's border leaves partial results, which a second launch adds in
// CTA order: no atomics, results do not depend on timing.
//
// Per tile and warp, with N = 8·NT query rows as the N side of m16n8k16:
//   Sᵀ[16 tokens × N] = K·Qᵀ          A = K rows,  B = Qᵀ
//   Oᵀ[d × N]        += Vᵀ·Pᵀ         A = Vᵀ,      B = Pᵀ (8×8 transposes)
// The query rows sit on the N side because a group has 1 to 16 heads: with
// them as M, at least half of every product would be padding.  p is split into
// three bf16 parts (3 × 8 bits: exact), so p·v has fp32's precision although
// the products run on the bf16 tensor path; that costs 16 more products per
// tile and stays far below the time the tile's bytes take.
//
// bf16 is bound by HBM, 512 bytes per (token, KV head): 4 sequences of 131,072
// tokens with 8 KV heads of 4 query heads take 322 us, 6.66 TB/s, as fast as the
// measured copy (6.55); 64 ragged ones of 4k to 16k tokens 402 us, 6.63 TB/s.
// 4 bits need 136 bytes and are bound by issue: the same contexts take 178 us,
// 3.2 TB/s (0.49), at 426 warp instructions per tile (88 to unpack codes, 33
// tensor products, 32 adds of products, the softmax and its three-part weights)
// and 0.6 issued per cycle and scheduler; all of this with up to 8 query rows.
// Short calls are bound by fetching their code, and by the chain of dependent
// steps from the lengths to the merge: 14 us for 2k tokens.
#include <cuda.h>

#include <atomic>

#include "q4.cuh"

namespace ekv {

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
constexpr int kModCtas = 296;     // two resident CTAs on each of 148 SMs: one wave
constexpr float kGrow = 8.0f;     // a score may pass the reference maximum by 2^8 before the state is rescaled
constexpr float kHuge = 3.402823466e38f;  // the largest finite number
constexpr float kNoMax = -kHuge;  // before the first score

struct ModArgs {
  const int32_t* page_table;
  const int32_t* seq_lens;
  const bf16* q;
  const int32_t* sel;
  const int32_t* n_sel;
  const float* slopes;
  const int32_t* prefix_lens;
  const int32_t* starts;
  const unsigned char* pool;  // 4-bit records
  float* out;
  float* lse;
  float* part;   // [2·CTAs, rows, D] partial p·v: slot 2c the first unit of CTA c, 2c + 1 its last
  float2* ml;    // [2·CTAs, rows] (maximum, sum) of a partial, in base 2
  int2* ref;     // [2·CTAs] positions that the bias of a partial is measured from
  int4* cut;     // [CTAs] the unit that starts in CTA c and is cut: (unit, first slot, pieces, −)
  float scale2;  // scale·log2(e), the factor of q·k without a cap
  float capx;    // scale/softcap
  float cap2;    // softcap·log2(e); 0: no cap
  int window, batch, Hkv, Hq, G, gsh, T, S,  // G = 1 << gsh
      num_phys, max_pages, cap;
  int min_tiles;    // the smallest run of a CTA: a step of every warp, for 4 bits of half of them
  int slack_tiles;  // how much longer a run may get where no CTA then crosses units: about the time of a crossing
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh(x) for |x| ≤ 1: the fifth convergent of Lambert's continued fraction,
// off by x¹¹/9.8e6 at most.  Scores under their cap lie there.
__device__ __forceinline__ float tanh_small(float x) {
  const float x2 = x * x;
  return __fdividef(x * fmaf(x2, x2 + 105.f, 945.f), fmaf(x2, fmaf(x2, 15.f, 420.f), 945.f));
}
// tanh(x) for any x: above 1 (e^2x − 1)/(e^2x + 1), where nothing cancels.
__device__ __forceinline__ float tanh_f32(float x) {
  const float ax = fabsf(x), e = ex2(fminf(ax, 15.f) * (2.f * kLog2e));
  const float t = copysignf(__fdividef(e - 1.f, e + 1.f), x);
  return ax > 1.f ? t : tanh_small(x);  // NaN: the second
}

// d = A·B + c on m16n8k16 bf16 (fragments as mma_bf16 in common.cuh).  d and c
// apart, and no volatile: the compiler is free to interleave products.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2], float c0, float c1,
                                    float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2],
                                    const float (&c)[4]) {
  mma(d, a, b, c[0], c[1], c[2], c[3]);
}
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  mma(d, a, b, 0.f, 0.f, 0.f, 0.f);
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ void tma_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}

// What one sequence lets its queries see, as tiles: nA from tile a0, then from
// tile b0 (a prefix, and the window behind it).
struct Visible {
  int L, start, prefix, a0, nA, b0, n;
};

struct Bounds {  // what the call says of one sequence
  int L, start, prefix;
};
__device__ __forceinline__ Bounds load_bounds(const ModArgs& a, int b) {
  return Bounds{a.seq_lens[b], a.starts ? a.starts[b] : 0, a.prefix_lens ? a.prefix_lens[b] : 0};
}
__device__ __forceinline__ Visible visible_tiles(const ModArgs& a, Bounds s) {
  Visible v;
  const int most = a.max_pages * a.S;
  if (s.L < 0 || s.L > most) {
    raise_flag(EKV_EFLAG_BAD_LEN);
    s.L = s.L < 0 ? 0 : most;
  }
  v.L = s.L;
  v.start = max(0, s.start);
  v.prefix = max(0, min(s.prefix, s.L));
  v.a0 = v.nA = v.b0 = v.n = 0;
  if (v.start >= v.L) return v;
  int lo = v.start;
  if (a.window > 0 && a.window < v.L) lo = max(lo, v.L - a.T - a.window + 1);  // a longer one hides nothing
  const int t_end = (v.L + kTile - 1) / kTile;
  v.b0 = lo / kTile;
  if (v.prefix > v.start && lo > v.start) {
    v.a0 = v.start / kTile;
    v.nA = min((v.prefix + kTile - 1) / kTile, v.b0) - v.a0;
    if (v.nA < 0) v.nA = 0;
  }
  v.n = v.nA + t_end - v.b0;
  return v;
}

// Tiles of one entry of the work list's outer level: a unit when pages are
// selected, else a sequence's count per KV head.  At least one: a unit that
// sees nothing gets one empty tile, which writes its rows.
__device__ __forceinline__ int selected_tiles(const ModArgs& a, int n_sel) {
  return max(1, max(0, min(n_sel, a.cap)) * (a.S / kTile));
}
__device__ __forceinline__ int group_tiles(const ModArgs& a, int grp) {
  return a.sel ? selected_tiles(a, a.n_sel[grp]) : max(1, visible_tiles(a, load_bounds(a, grp)).n);
}

// Pieces of about 1/inv tiles that a unit of n tiles is cut into: at least one,
// at most n, the same for everybody who asks.
__device__ __forceinline__ int piece_count(int n, float inv) {
  return min(n, 1 + static_cast<int>(static_cast<float>(n - 1) * inv));
}

// The part of a unit that a CTA works on: tiles t0 .. t1−1 of n, one of
// `pieces` parts (the first one of them knows how many).
struct Segment {
  Visible vis;
  int unit, b, h, t0, t1, n, pieces;
};

// The physical place of a tile (row of the pools, or record of the 4-bit pool)
// and the position of its first token, a multiple of 16; bit 0 of j0 says that
// every row sees all of it, so that most tiles need no masks, bit 1 that it lies
// behind every row.  at = −1: nothing there to see, and a position that no mask
// lets through.
struct Tile {
  int at, j0;
};

__device__ __forceinline__ Tile resolve_tile(const ModArgs& a, const Segment& s, int t) {
  Tile r{-1, -kTile};
  if (t < s.t0 || s.vis.n == 0) return r;
  const int sh = a.S == kTile ? 0 : 1, tpp = 1 << sh;  // tiles of a page: 1 or 2
  int lp, part;
  if (a.sel == nullptr) {
    const int tile = t < s.vis.nA ? s.vis.a0 + t : s.vis.b0 + t - s.vis.nA;
    lp = tile >> sh;
    part = tile & (tpp - 1);
  } else {
    const int slot = t >> sh;
    part = t & (tpp - 1);
    if (slot >= max(0, min(a.n_sel[s.unit], a.cap))) return r;  // the empty unit's tile
    lp = a.sel[static_cast<size_t>(s.unit) * a.cap + slot];
    if (lp < 0 || lp >= (s.vis.L + a.S - 1) / a.S) {
      raise_flag(EKV_EFLAG_BAD_SEL);
      return r;
    }
  }
  const int j0 = lp * a.S + part * kTile;
  if (a.sel != nullptr) {  // a page may hold no visible tile
    const int tile = j0 / kTile;
    const bool in_b = tile >= s.vis.b0 && j0 < s.vis.L;
    const bool in_a = tile >= s.vis.a0 && tile < s.vis.a0 + s.vis.nA;
    if (!in_a && !in_b) return r;
  }
  const int phys = a.page_table[static_cast<size_t>(s.b) * a.max_pages + lp];
  if (!phys_ok(phys, a.num_phys)) return r;
  r.at = (phys * a.Hkv + s.h) * tpp + part;
  // (a prefix hides nothing from any row at or behind position 0: with L < T some lie before it)
  const bool whole = j0 >= s.vis.start &&
                     ((j0 + kTile <= s.vis.prefix && s.vis.L >= a.T) ||
                      (j0 + kTile <= s.vis.L - a.T + 1 && (a.window <= 0 || s.vis.L - 1 - j0 < a.window)));
  r.j0 = j0 | (whole ? 1 : 0) | (j0 + kTile <= s.vis.L - a.T + 1 ? 2 : 0);
  return r;
}

// Position of a segment's first (last) tile, whether or not it can be read.
__device__ __forceinline__ int tile_position(const ModArgs& a, const Segment& s, int t) {
  const int sh = a.S == kTile ? 0 : 1;
  if (s.vis.n == 0) return 0;
  if (a.sel == nullptr) return (t < s.vis.nA ? s.vis.a0 + t : s.vis.b0 + t - s.vis.nA) * kTile;
  const int slot = t >> sh;
  if (slot >= max(0, min(a.n_sel[s.unit], a.cap))) return 0;
  const int lp = a.sel[static_cast<size_t>(s.unit) * a.cap + slot];
  return lp < 0 || lp >= a.max_pages ? 0 : lp * a.S + (t - (slot << sh)) * kTile;
}

// The distance that the bias of a piece is measured from, so that far tokens
// keep their differences in fp32: the nearest one for a falling bias, the
// farthest for a rising one.  Any value is right; this one is precise.
__device__ __forceinline__ int ref_distance(float slope, int i, int2 ref) {
  return slope >= 0.f ? max(0, i - ref.y) : abs(i - ref.x);
}

// Where a CTA's run of the work list starts, and how the list is cut.
struct Run {
  long long total;   // tiles of the list
  long long start;   // the run's first tile, or its piece when the cuts are aligned
  long long grp_at;  // the first of group grp, in the same count
  int per;           // tiles of a run, about those of a piece
  int grp, grp_tiles;  // the group that holds the start (−1: no such run), tiles of each of its units
  bool aligned;
};

// Cutting the list into equal runs keeps every CTA equally busy but lets one
// cross units, which costs it a second set of queries and a second merge;
// cutting every unit into equal pieces costs nothing while there are CTAs
// enough, so that comes first.  Every warp works it out by itself, N groups per
// lane at a time, all their loads first (block-wide scans took 2.4 us of a 24 us
// call, loads one by one 1.9 of 15).  N = 1: at most 32 groups, without loops; short
// calls wait for instructions as much as for data, and the same code with N = 4
// took 0.5 us more of 10 to 20.
template <int N>
__device__ __forceinline__ Run find_run(const ModArgs& a, int groups, int mult) {
  constexpr int kChunk = 32 * N;
  const int lane = threadIdx.x & 31, bound = N == 1 ? 1 : groups;
  Run run;
  int mine[N];  // tiles of groups 32·i + lane of the chunk in work
  int held = -1;
  auto load_chunk = [&](int c0) {
    if (held == c0) return;
    held = c0;
    Bounds s[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (N > 1 && c0 + 32 * i >= groups) continue;
      const int grp = min(c0 + 32 * i + lane, groups - 1);
      if (a.sel) s[i].L = a.n_sel[grp];
      else s[i] = load_bounds(a, grp);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      mine[i] = c0 + 32 * i + lane >= groups ? 0
                : a.sel                      ? selected_tiles(a, s[i].L)
                                             : max(1, visible_tiles(a, s[i]).n);
  };
  auto sum_over_groups = [&](auto value) {  // value(tiles), times the units of a group
    long long total = 0;
    for (int c0 = 0; c0 < bound; c0 += kChunk) {
      load_chunk(c0);
      int x = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) x += value(mine[i]);
      // in two halves: 128 long sequences pass 32 bits
      total += (__reduce_add_sync(0xffffffffu, x & 0xffff) +
                (static_cast<long long>(__reduce_add_sync(0xffffffffu, x >> 16)) << 16)) * mult;
    }
    return total;
  };
  const long long total = run.total = sum_over_groups([](int n) { return n; });
  const int ctas = static_cast<int>(gridDim.x);
  int per = total < 0x70000000 ? static_cast<int>((static_cast<uint32_t>(total) + ctas - 1) / static_cast<uint32_t>(ctas))
                               : static_cast<int>((total + ctas - 1) / ctas);
  per = max(per, a.min_tiles);
  bool aligned = false;
  if (static_cast<long long>(groups) * mult <= ctas) {
    auto fits = [&](int by) {
      const float inv = 1.f / static_cast<float>(by);
      return sum_over_groups([inv](int n) { return n > 0 ? piece_count(n, inv) : 0; }) <= ctas;
    };
    // what the CTAs of one of equal units would take; else the equal run
    const float units = static_cast<float>(groups * mult);
    const float each = floorf(static_cast<float>(ctas) / units + 1e-3f);
    const int by = max(a.min_tiles, static_cast<int>(ceilf(static_cast<float>(total) / (units * each))));
    if (by - per <= a.slack_tiles && fits(by)) {
      aligned = true;
      per = by;
    } else {
      aligned = by != per && fits(per);
    }
  }
  run.aligned = aligned;
  run.per = per;
  // the group that holds this CTA's start: counted in pieces, or in tiles
  run.start = aligned ? blockIdx.x : static_cast<long long>(per) * blockIdx.x;
  const float inv_per = 1.f / static_cast<float>(per);
  run.grp_at = 0;
  run.grp = -1;
  run.grp_tiles = 0;
  for (int c0 = 0; c0 < bound && run.grp < 0; c0 += kChunk) {
    load_chunk(c0);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (N > 1 && (run.grp >= 0 || c0 + 32 * i >= groups)) continue;
      const int len = (aligned && mine[i] > 0 ? piece_count(mine[i], inv_per) : mine[i]) * mult;
      int up = len;  // inclusive scan over the lanes
#pragma unroll
      for (int sh = 1; sh < 32; sh <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, up, sh);
        if (lane >= sh) up += y;
      }
      const int off = run.start - run.grp_at < 0x7fffffff ? static_cast<int>(run.start - run.grp_at) : 0x7fffffff;
      const uint32_t hit = __ballot_sync(0xffffffffu, up - len <= off && off < up);
      if (hit) {
        const int from = __ffs(hit) - 1;
        run.grp = c0 + 32 * i + from;
        run.grp_tiles = __shfl_sync(0xffffffffu, mine[i], from);
        run.grp_at += __shfl_sync(0xffffffffu, up - len, from);
      } else {
        run.grp_at += __shfl_sync(0xffffffffu, up, 31);
      }
    }
  }
  return run;
}

// NT: groups of 8 query rows per warp.  4 bits at NT = 1: eight warps of at most
// 128 registers and two tiles a step, since turning codes into numbers keeps the
// issue slots busy and what is done once per step counts; on 4 × 131,072 tokens 16
// warps per SM with two tiles take 179 us, 20 with one 199, 12 with two and no
// spills 190.  Else four warps and one tile, where copies alone bound the step.
template <int D, int NT, bool Q4>
struct Shape {
  static constexpr int NW = Q4 && NT == 1 ? 8 : 4;  // warps of a CTA
  static constexpr int U = Q4 && NT == 1 ? 2 : 1;   // tiles of a step
  static constexpr int tile_bytes = Q4 ? q4_record_bytes(D) : 2 * kTile * D * 2;
  static constexpr int slot_bytes = U * ((tile_bytes + 127) / 128 * 128);
  static constexpr int threads = 32 * NW;
};

// Floats from one row of the merge buffer to the next, and where number d of a
// row lies: 2·pitch is 8 or 24 mod 32, and the 4-bit lanes' shares of D/8
// numbers are one apart, so that the warps' stores meet no bank twice.
constexpr int merge_pitch(int d, bool q4) { return q4 ? d + 12 : d + 4; }
template <int D, bool Q4>
__device__ __forceinline__ int merge_at(int d) {
  return Q4 ? d + d / (D / 8) : d;
}

template <int D, int NT, int R, bool Q4>
constexpr int mod_stages() {
  // as many copies in flight as two CTAs' shared memory holds beside the merge buffer
  using Sh = Shape<D, NT, Q4>;
  constexpr int merge = (Sh::NW * 8 * NT) * merge_pitch(D, Q4) * 4;
  constexpr int room = 112 * 1024 - merge;
  constexpr int n = room / (Sh::NW / R * Sh::slot_bytes);
  return n > 6 ? 6 : n;
}

template <int D, int NT, int R, bool Q4>
constexpr size_t mod_smem() {
  using Sh = Shape<D, NT, Q4>;
  return 1024 + static_cast<size_t>(Sh::NW / R) * mod_stages<D, NT, R, Q4>() * Sh::slot_bytes +
         static_cast<size_t>(Sh::NW * 8 * NT) * merge_pitch(D, Q4) * 4;
}

// R: warps that share a tile stream, each with its own rows (8·NT·R ≥ G·T).
template <int D, int NT, int R, bool Q4>
__global__ void __launch_bounds__(Shape<D, NT, Q4>::threads, 2)
    mod_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, ModArgs a) {
  using Sh = Shape<D, NT, Q4>;
  constexpr int NW = Sh::NW, U = Sh::U, NS = NW / R, ST = mod_stages<D, NT, R, Q4>();
  constexpr int KS = D / 16, MT = D / 16, PITCH = merge_pitch(D, Q4);
  static_assert(ST >= 2 && NW % R == 0, "ring too small");
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint64_t bars[NS * ST];
  __shared__ float s_m[NW][8 * NT], s_l[NW][8 * NT], s_c[NW][8 * NT];
  __shared__ float2 s_row[8 * NT * R];  // what a row's sums are multiplied by, and what is added before
  constexpr bool kSharedQ = Q4 && NT == 1;  // one set of query fragments for all warps, to spare registers
  __shared__ uint2 s_q[kSharedQ ? KS : 1][32];
  __shared__ Segment s_seg[2];  // the unit in work, and the next

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const int stream = warp / R, rg = warp - stream * R;
  // the ring starts on a 1024-byte boundary: the 128-byte swizzle repeats every 8 rows
  unsigned char* ring = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  float* red = reinterpret_cast<float*>(ring + NS * ST * Sh::slot_bytes);
  if (tid < NS * ST) {
    mbar_init(&bars[tid], U);  // an arrival per tile
    fence_mbar_init();
  }
  if (!Q4 && tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
  }
  grid_dep_enter();

  // this CTA's run of the work list
  const int mult = a.sel ? 1 : a.Hkv, groups = a.sel ? a.batch * a.Hkv : a.batch;
  if (tid == 0) a.cut[blockIdx.x] = make_int4(0, 0, 0, 0);
  const Run run = groups <= 32 ? find_run<1>(a, groups, mult) : find_run<4>(a, groups, mult);
  const bool aligned = run.aligned;
  const long long total = run.total;
  const int per = run.per;
  const float inv_per = 1.f / static_cast<float>(per);
  long long pos = run.start, grp_at = run.grp_at;
  int grp = run.grp;
  const int grp_tiles = run.grp_tiles;
  if (grp < 0) return;  // more CTAs than runs
  const long long end = pos + per < total ? pos + per : total;  // of a run of tiles

  Segment seg;  // the next one to work on; s_seg holds the one in work
  seg.vis = visible_tiles(a, load_bounds(a, a.sel ? grp / a.Hkv : grp));
  seg.n = grp_tiles;
  auto place = [&]() {  // the unit at pos of group grp
    const uint32_t off = static_cast<uint32_t>(pos - grp_at);
    seg.b = a.sel ? grp / a.Hkv : grp;
    int hh;
    if (aligned) {
      // pieces of equal length, the first n mod np of them one longer
      const uint32_t np = static_cast<uint32_t>(piece_count(seg.n, inv_per)), unit = off / np;
      const int piece = static_cast<int>(off - unit * np), each = static_cast<int>(seg.n / np);
      const int more = seg.n - each * static_cast<int>(np);
      hh = static_cast<int>(unit);
      seg.t0 = piece * each + min(piece, more);
      seg.t1 = seg.t0 + each + (piece < more ? 1 : 0);
      seg.pieces = static_cast<int>(np);
    } else {
      hh = static_cast<int>(off / static_cast<uint32_t>(seg.n));
      seg.t0 = static_cast<int>(off) - hh * seg.n;
      const long long left = end - pos;
      seg.t1 = left < seg.n - seg.t0 ? seg.t0 + static_cast<int>(left) : seg.n;
      seg.pieces = static_cast<int>((pos - seg.t0 + seg.n - 1) / per) - static_cast<int>(blockIdx.x) + 1;
    }
    seg.h = a.sel ? grp % a.Hkv : hh;
    seg.unit = seg.b * a.Hkv + seg.h;
  };

  unsigned char* my_ring = ring + stream * ST * Sh::slot_bytes;
  uint64_t* my_bar = bars + stream * ST;
  int ring_at = 0;            // the slot whose turn it is
  unsigned int parity = 0;    // and its barrier's phase
  Tile cur, nxt;
  // One tile into its place of slot sl, by the lane that looked it up: a step's
  // copies start side by side, and no lane has to be told another's tile.
  auto issue = [&](const Tile& x, int sl, int u) {
    if (x.at < 0) {
      mbar_arrive(&my_bar[sl]);
      return;
    }
    unsigned char* dst = my_ring + sl * Sh::slot_bytes + u * (Sh::slot_bytes / U);
    mbar_arrive_expect_tx(&my_bar[sl], Sh::tile_bytes);
    if constexpr (Q4) {
      bulk_g2s(dst, a.pool + static_cast<size_t>(x.at) * Sh::tile_bytes, Sh::tile_bytes, &my_bar[sl]);
    } else {
#pragma unroll
      for (int half = 0; half < D / 64; ++half) {
        tma_2d(dst + half * kTile * 128, &kmap, half * 64, x.at * kTile, &my_bar[sl]);
        tma_2d(dst + (D / 64 + half) * kTile * 128, &vmap, half * 64, x.at * kTile, &my_bar[sl]);
      }
    }
  };
  // A stream's step k is tiles U·(stream + NS·k) .. + U − 1 of the segment, counted
  // from its end: under a bias that falls with distance the nearest tokens hold
  // the largest scores, and the reference maximum then hardly ever moves (from the
  // other end it moved at 62% of all steps).  A lookup resolves the 32 tiles of
  // 32/U steps, one per lane.
  constexpr int kSteps = 32 / U;
  auto stream_steps = [&](const Segment& s) {
    const int n = s.t1 - s.t0 - U * stream;
    return n > 0 ? (n + U * NS - 1) / (U * NS) : 0;
  };
  auto lookup = [&](const Segment& s, int batch) {
    return resolve_tile(a, s, s.t1 - 1 - (U * (stream + NS * (kSteps * batch + lane / U)) + lane % U));
  };
  const int rows = a.G * a.T;
  // a lane's share of its query row (row g of each group of 8): bf16 caches, the
  // B fragments; 4 bits, D/4 numbers from D/4·t4
  uint32_t q_raw[NT][KS * 2];
  // The unit's queries and first copies are on their way.  used: the slots have been
  // read, and written where masked rows of V were zeroed, since the kernel's start;
  // that comes before the copies into them.
  auto prologue = [&](const Segment& s, bool used) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = (rg * NT + nt) * 8 + g, rr = row < rows ? row : 0, t = rr >> a.gsh;
      const bf16* qp = a.q + ((static_cast<size_t>(s.b) * a.T + t) * a.Hq + s.h * a.G + rr - t * a.G) * D;
      if constexpr (Q4) {
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          const uint4 x = *reinterpret_cast<const uint4*>(qp + D / 4 * t4 + 8 * w);
          q_raw[nt][4 * w] = x.x;
          q_raw[nt][4 * w + 1] = x.y;
          q_raw[nt][4 * w + 2] = x.z;
          q_raw[nt][4 * w + 3] = x.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < KS * 2; ++i) q_raw[nt][i] = *reinterpret_cast<const uint32_t*>(qp + 8 * i + 2 * t4);
      }
    }
    const int nk = stream_steps(s);
    cur = lookup(s, 0);
    const int step = lane / U, sl = ring_at + step < ST ? ring_at + step : ring_at + step - ST;
    if (rg == 0 && step < ST && step < nk) {
      if (used) fence_proxy_async_shared();
      issue(cur, sl, lane % U);
    }
    if (nk > kSteps - ST) nxt = lookup(s, 1);
  };
  auto stream_sync = [&]() {
    if constexpr (R == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + stream), "r"(32 * R) : "memory");
  };

  place();
  bool first_segment = true;
  int which = 0;
  __syncthreads();  // barriers initialised
  prologue(seg, false);
  if (tid == 0) s_seg[0] = seg;
  __syncthreads();

  for (;;) {
    const Segment& now = s_seg[which];
    // ---- the unit's queries
    int qd[NT][2];  // the lane's columns (rows 2·t4, 2·t4 + 1 of each group of 8): position − reference distance − g
    float slope2[NT][2];
    int2 ref = make_int2(0, 0);
    if (a.slopes) ref = make_int2(tile_position(a, now, now.t0), tile_position(a, now, now.t1 - 1) + kTile - 1);
    uint32_t qf[kSharedQ ? 1 : KS][NT][2];
    float qsum[NT][2], qdown[NT][2], qc[NT][4];  // 4 bits, the lane's columns: (Σ q)·factor, factor/2^k, −8·Σ q·2^k (twice)
    auto row_position = [&](int nt, int e) {
      const int row = (rg * NT + nt) * 8 + 2 * t4 + e;
      return now.vis.L - a.T + ((row < rows ? row : 0) >> a.gsh);
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        slope2[nt][e] = 0.f;
        qd[nt][e] = 0;
        if (a.slopes) {
          const int row = (rg * NT + nt) * 8 + 2 * t4 + e, rr = row < rows ? row : 0;
          const float sl = a.slopes[now.h * a.G + (rr & (a.G - 1))];
          const int i = row_position(nt, e);
          slope2[nt][e] = sl * kLog2e;
          qd[nt][e] = i - ref_distance(sl, i, ref) - g;
        }
      }
      if constexpr (!Q4) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          qf[ks][nt][0] = q_raw[nt][2 * ks];
          qf[ks][nt][1] = q_raw[nt][2 * ks + 1];
        }
      } else {
        // Scaled by a power of two to a largest number near 2^120 (exact: the codes
        // enter as subnormals n·2⁻¹³³, so sums of products stay below 1).  Word w of
        // the lane's share gives the pairs (8w + i, 8w + i + 4), as the codes do; codes
        // at odd i come 16 times too large, so their numbers are divided by 16.
        float sum = 0.f, top = 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const float lo = bf16_lo(q_raw[nt][i]), hi = bf16_hi(q_raw[nt][i]);
          sum += lo + hi;
          top = fmaxf(top, fmaxf(fabsf(lo), fabsf(hi)));
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int k = 120 + 127 - static_cast<int>(__float_as_uint(top) >> 23);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + max(-126, min(126, k))) << 23);
        uint32_t qh[KS][2];
#pragma unroll
        for (int w = 0; w < D / 32; ++w)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float by = (i & 1) ? up * 0.0625f : up;
            const uint32_t x = q_raw[nt][4 * w + (i >> 1)], y = q_raw[nt][4 * w + 2 + (i >> 1)];
            qh[2 * w + (i >> 1)][i & 1] = (i & 1) ? pack_bf16_exact(bf16_hi(x) * by, bf16_hi(y) * by)
                                                  : pack_bf16_exact(bf16_lo(x) * by, bf16_lo(y) * by);
          }
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          if constexpr (kSharedQ) {
            if (warp == 0) s_q[ks][lane] = make_uint2(qh[ks][0], qh[ks][1]);
          } else {
            qf[ks][nt][0] = qh[ks][0];
            qf[ks][nt][1] = qh[ks][1];
          }
        }
        // zf·2^133/up: a factor past the ends of fp32 (tiny caps, zero queries) stays
        // finite, since it may meet a sum or a step of 0
        const float zf = a.cap2 != 0.f ? a.capx : a.scale2;
        const float down = fminf(kHuge, zf * (0x1p66f / up) * 0x1p67f);
        const float qs = fabsf(sum) <= kHuge ? fmaxf(-kHuge, fminf(kHuge, sum * zf)) : sum;
        qsum[nt][0] = __shfl_sync(0xffffffffu, qs, 8 * t4);
        qsum[nt][1] = __shfl_sync(0xffffffffu, qs, 8 * t4 + 4);
        const float c8 = sum * (up * -0x1p-65f) * 0x1p-65f;
        qc[nt][0] = qc[nt][2] = __shfl_sync(0xffffffffu, c8, 8 * t4);
        qc[nt][1] = qc[nt][3] = __shfl_sync(0xffffffffu, c8, 8 * t4 + 4);
        qdown[nt][0] = __shfl_sync(0xffffffffu, down, 8 * t4);
        qdown[nt][1] = __shfl_sync(0xffffffffu, down, 8 * t4 + 4);
      }
    }

    float o[MT][NT][4], m[NT][2], l[NT][2], corr[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < MT; ++j) o[j][nt][0] = o[j][nt][1] = o[j][nt][2] = o[j][nt][3] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nt][e] = kNoMax;  // the reference maximum
        l[nt][e] = corr[nt][e] = 0.f;
      }
    }

    if constexpr (kSharedQ) __syncthreads();

    // ---- the tiles
    const int nk = stream_steps(now);
    for (int k = 0; k < nk; ++k) {
      const int in = k & (kSteps - 1);  // within the 32 tiles looked up
      if (k > 0 && in == 0) {
        cur = nxt;
        nxt = lookup(now, k / kSteps + 1);
      }
      int j0[U];
#pragma unroll
      for (int u = 0; u < U; ++u) j0[u] = __shfl_sync(0xffffffffu, cur.j0, in * U + u);
      const int sl = ring_at;
      if (!mbar_wait(&my_bar[sl], parity)) mbar_wait(&my_bar[sl], parity);
      unsigned char* const buf = my_ring + sl * Sh::slot_bytes;
      int flags = 3;
#pragma unroll
      for (int u = 0; u < U; ++u) flags &= j0[u];
      const bool whole = flags & 1;

      // scores: Sᵀ of the step's tiles, in base 2 when there is no cap, else over the cap
      float z[U][NT][4];
      if constexpr (!Q4) {
        float z2[NT][4];
        const uint32_t kbase = smem_addr(buf);
        const int tok = lane & 15, ch = lane >> 4;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const int c = 2 * ks + ch;
          uint32_t af[4];
          ldsm_x4(kbase + (c >> 3) * (kTile * 128) + tok * 128 + (((c & 7) ^ (tok & 7)) << 4), af);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float(&to)[4] = ks & 1 ? z2[nt] : z[0][nt];
            if (ks < 2) mma_first(to, af, qf[ks][nt]);
            else mma(to, af, qf[ks][nt], to);
          }
        }
        const float zf = a.cap2 != 0.f ? a.capx : a.scale2;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) z[0][nt][e] = (z[0][nt][e] + z2[nt][e]) * zf;
      } else {
        uint32_t w0[U][D / 32], w1[U][D / 32];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const unsigned char* k0 = buf + u * (Sh::slot_bytes / U) + g * (D / 2) + t4 * (D / 8);
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(k0), y = *reinterpret_cast<const uint4*>(k0 + 8 * (D / 2));
            w0[u][0] = x.x; w0[u][1] = x.y; w0[u][2] = x.z; w0[u][3] = x.w;
            w1[u][0] = y.x; w1[u][1] = y.y; w1[u][2] = y.z; w1[u][3] = y.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(k0), y = *reinterpret_cast<const uint2*>(k0 + 8 * (D / 2));
            w0[u][0] = x.x; w0[u][1] = x.y;
            w1[u][0] = y.x; w1[u][1] = y.y;
          }
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w)
#pragma unroll
          for (int b = 0; b < 2; ++b) {  // codes 0, 1, 4, 5 of a word, then 2, 3, 6, 7
            uint32_t bq[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if constexpr (kSharedQ) {
                const uint2 x = s_q[2 * w + b][lane];
                bq[nt][0] = x.x;
                bq[nt][1] = x.y;
              } else {
                bq[nt][0] = qf[2 * w + b][nt][0];
                bq[nt][1] = qf[2 * w + b][nt][1];
              }
            }
            // As bf16, 0x000n is the subnormal n·2⁻¹³³ and 0x00n0 is 16n·2⁻¹³³ (exponent
            // field 1 has the subnormals' spacing): a code in the low byte of a half
            // is a number already.  (fp16 would do too, but the tensor cores align sums
            // by exponent fields: there the products lost three bits more.)
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const uint32_t x = w0[u][w] >> (8 * b), y = w1[u][w] >> (8 * b);
              const uint32_t af[4] = {x & 0x000f000fu, y & 0x000f000fu, x & 0x00f000f0u, y & 0x00f000f0u};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                // from −8·Σ q: the sum is of n − 8, which keeps it small
                if (w + b == 0) mma(z[u][nt], af, bq[nt], qc[nt]);
                else mma(z[u][nt], af, bq[nt], z[u][nt]);
              }
            }
          }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t* pairs = reinterpret_cast<const uint32_t*>(buf + u * (Sh::slot_bytes / U) + 16 * D);
          const uint32_t ka = pairs[g], kb = pairs[g + 8];
          const float ks0 = bf16_lo(ka), ks1 = bf16_lo(kb);
          const float kz0 = fmaf(8.f, ks0, bf16_hi(ka)), kz1 = fmaf(8.f, ks1, bf16_hi(kb));  // the value of code 8
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              z[u][nt][e] = fmaf(ks0, z[u][nt][e] * qdown[nt][e], kz0 * qsum[nt][e]);
              z[u][nt][2 + e] = fmaf(ks1, z[u][nt][2 + e] * qdown[nt][e], kz1 * qsum[nt][e]);
            }
        }
      }
      if (a.cap2 != 0.f) {
        bool large = false;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) large |= fabsf(z[u][nt][e]) > 1.f;
        if (__any_sync(0xffffffffu, large)) {
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) z[u][nt][e] = a.cap2 * tanh_f32(z[u][nt][e]);
        } else {  // 8 instructions a score in place of 20
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) z[u][nt][e] = a.cap2 * tanh_small(z[u][nt][e]);
        }
      }
      if (a.slopes) {
        if (flags & 2) {  // behind the query the bias is linear
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float at = static_cast<float>(qd[nt][e] - (j0[u] & -kTile));
                z[u][nt][e] = fmaf(-slope2[nt][e], at, z[u][nt][e]);
                z[u][nt][2 + e] = fmaf(-slope2[nt][e], at - 8.f, z[u][nt][2 + e]);
              }
        } else {
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int i = row_position(nt, e), d0 = i - g - qd[nt][e], off = i - (j0[u] & -kTile) - g;
                z[u][nt][e] = fmaf(-slope2[nt][e], static_cast<float>(abs(off) - d0), z[u][nt][e]);
                z[u][nt][2 + e] = fmaf(-slope2[nt][e], static_cast<float>(abs(off - 8) - d0), z[u][nt][2 + e]);
              }
        }
      }
      // masks: only steps that not every row sees whole
      uint32_t apart = 0;  // bf16: tokens that some rows see and others do not, with a V that is not finite
      if (!whole) {
        auto sees = [&](int i, int j) {
          return j >= now.vis.start && i >= 0 && j < now.vis.L &&
                 (j < now.vis.prefix || (j <= i && (a.window <= 0 || i - j < a.window)));
        };
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!sees(row_position(nt, e & 1), (j0[u] & -kTile) + g + (e >> 1) * 8)) z[u][nt][e] = -INFINITY;
        if constexpr (!Q4) {
          // 0·V must not turn a masked NaN into the sum: rows of V that nobody
          // sees are zeroed; a row only some see is set apart if it has one
          bool any = false, all = true;
          if (lane < kTile)
            for (int t = 0; t < a.T; ++t) {
              const bool v = sees(now.vis.L - a.T + t, (j0[0] & -kTile) + lane);
              any |= v;
              all &= v;
            }
          const uint32_t seen = __ballot_sync(0xffffffffu, any && lane < kTile);
          const uint32_t some = seen & ~__ballot_sync(0xffffffffu, all && lane < kTile);
          // lane: half a row (D/16 chunks of 16 bytes) of token lane/2
          const int tok = lane >> 1;
          unsigned char* row = buf + D / 64 * kTile * 128 + tok * 128;
          auto chunk = [&](int i) {
            const int c = (lane & 1) * (D / 16) + i;
            return reinterpret_cast<uint4*>(row + (c >> 3) * (kTile * 128) + (c & 7) * 16);
          };
          if (!(seen >> tok & 1u)) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) *chunk(i) = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_shared();  // these stores come before the copies that refill the slot
          }
          if (some) {
            bool bad = false;
            if (some >> tok & 1u) {
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                const uint4 x = *chunk(i);
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  bad |= (xs[e] & 0x7f80u) == 0x7f80u || (xs[e] & 0x7f800000u) == 0x7f800000u;
              }
            }
            const uint32_t lanes = __ballot_sync(0xffffffffu, bad);
            for (uint32_t rest = lanes; rest; rest &= rest - 1) apart |= 1u << ((__ffs(rest) - 1) >> 1);
          }
          __syncwarp();
        }
      }
      // A score far above the reference: new maxima, and the state follows.
      auto move_reference = [&](int nt, int e, float to) {
        if (to > m[nt][e]) {
          const float f = ex2(m[nt][e] - to);
          m[nt][e] = to;
          l[nt][e] *= f;
          corr[nt][e] *= f;
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            o[j][nt][e] *= f;
            o[j][nt][2 + e] *= f;
          }
        }
      };
      auto max_over_tokens = [&](float x) {
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
      };
      float w[U][NT][4];  // the weights of V: p, and for 4 bits p·step
      float vs[U][2], vmid[U][2];  // 4 bits: V's step and the value of code 8, of tokens g and g + 8
      if constexpr (!Q4) {
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) grow |= z[0][nt][e] > m[nt][e & 1] + kGrow;
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) move_reference(nt, e, max_over_tokens(fmaxf(z[0][nt][e], z[0][nt][2 + e])));
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            w[0][nt][e] = ex2(z[0][nt][e] - m[nt][e & 1]);
            l[nt][e & 1] += w[0][nt][e];
          }
      } else {
        // w = p·step·2^64, since the codes of V enter as bf16 subnormals n·2⁻¹³³.  The
        // reference follows p·step and p·(the value of code 8) as well as p, so that w
        // and both sums stay in their range whatever the steps and values: it is the
        // largest score plus the largest of log2(step), log2|value| − 64 and −32.
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t* pairs = reinterpret_cast<const uint32_t*>(buf + u * (Sh::slot_bytes / U) + 16 * D);
          const uint32_t va = pairs[16 + g], vb = pairs[24 + g];
          vs[u][0] = bf16_lo(va);
          vs[u][1] = bf16_lo(vb);
          vmid[u][0] = fmaf(8.f, vs[u][0], bf16_hi(va));
          vmid[u][1] = fmaf(8.f, vs[u][1], bf16_hi(vb));
        }
        if (!whole) {
          // A masked token's pair may hold anything, and 0·NaN must not reach the
          // sums: it counts as 0 where none of the lane's rows sees the token; a row
          // that does see one that is not finite gets its NaN through the score.
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              bool seen = false;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) seen |= z[u][nt][2 * t + e] != -INFINITY;
              if (!seen || !(fabsf(vs[u][t]) < 0x1p63f && fabsf(vmid[u][t]) < INFINITY)) {
                vs[u][t] = vmid[u][t] = 0.f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int e = 0; e < 2; ++e)
                    if (z[u][nt][2 * t + e] != -INFINITY) z[u][nt][2 * t + e] = NAN;
              }
            }
        }
        float sum[NT][2], mid[NT][2];
        auto weigh = [&]() {
          bool fits = true;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              sum[nt][e] = l[nt][e];
              mid[nt][e] = corr[nt][e];
#pragma unroll
              for (int u = 0; u < U; ++u)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                  const float p = ex2(z[u][nt][2 * t + e] - m[nt][e]);
                  sum[nt][e] += p;
                  mid[nt][e] = fmaf(p, vmid[u][t], mid[nt][e]);
                  w[u][nt][2 * t + e] = p * (vs[u][t] * 0x1p64f);
                  fits = fits && w[u][nt][2 * t + e] <= 0x1p100f;
                }
              fits = fits && sum[nt][e] <= 0x1p100f && fabsf(mid[nt][e]) <= 0x1p100f;
            }
          return fits;
        };
        if (__any_sync(0xffffffffu, !weigh())) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float top = -INFINITY;
#pragma unroll
              for (int u = 0; u < U; ++u)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                  const float x = z[u][nt][2 * t + e];
                  const float size = fmaxf(__log2f(vs[u][t]), __log2f(fabsf(vmid[u][t])) - 64.f);
                  if (x > -INFINITY) top = fmaxf(top, x + fminf(64.f, fmaxf(-32.f, size)));
                }
              move_reference(nt, e, max_over_tokens(top));
            }
          weigh();
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            l[nt][e] = sum[nt][e];
            corr[nt][e] = mid[nt][e];
          }
      }
      // w in three bf16 parts, as B fragments
      uint32_t pf[U][NT][3][2];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if constexpr (!Q4) {
            if (apart) {
              // tokens set apart, by hand: only rows that see them, p > 0
              const unsigned char* vt = buf + D / 64 * kTile * 128;
              for (uint32_t rest = apart; rest; rest &= rest - 1) {
                const int tok = __ffs(rest) - 1, from = (tok & 7) * 4 + t4;
                const float pa = __shfl_sync(0xffffffffu, tok < 8 ? w[0][nt][0] : w[0][nt][2], from);
                const float pb = __shfl_sync(0xffffffffu, tok < 8 ? w[0][nt][1] : w[0][nt][3], from);
#pragma unroll
                for (int j = 0; j < MT; ++j)
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    const int col = 16 * j + 8 * e + g, c = (col & 63) >> 3;
                    const float v = __bfloat162float(*reinterpret_cast<const bf16*>(
                        vt + (col >> 6) * (kTile * 128) + tok * 128 + ((c ^ (tok & 7)) << 4) + (col & 7) * 2));
                    if (pa > 0.f) o[j][nt][2 * e] = fmaf(pa, v, o[j][nt][2 * e]);
                    if (pb > 0.f) o[j][nt][2 * e + 1] = fmaf(pb, v, o[j][nt][2 * e + 1]);
                  }
              }
            }
          }
          float(&x)[4] = w[u][nt];
#pragma unroll
          for (int part = 0; part < 3; ++part) {
            pf[u][nt][part][0] = transpose8x8(__byte_perm(__float_as_uint(x[0]), __float_as_uint(x[1]), 0x7632));
            pf[u][nt][part][1] = transpose8x8(__byte_perm(__float_as_uint(x[2]), __float_as_uint(x[3]), 0x7632));
            if (part < 2) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                x[e] -= __uint_as_float(__float_as_uint(x[e]) & 0xffff0000u);
                if (Q4 && part == 0) corr[nt][e & 1] = fmaf(-0x1p-61f, x[e], corr[nt][e & 1]);
              }
            }
          }
        }
      if constexpr (!Q4) {
        if (apart) {
          stream_sync();  // the warps that share the tile have all read the rows
          unsigned char* vt = buf + D / 64 * kTile * 128;
          for (uint32_t rest = apart; rest; rest &= rest - 1) {
            const int tok = __ffs(rest) - 1;
            if (lane < D / 8)
              *reinterpret_cast<uint4*>(vt + (lane >> 3) * (kTile * 128) + tok * 128 + (lane & 7) * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_shared();
          __syncwarp();
        }
      }
      // p·v.  The tensor cores drop bits when they add to an accumulator; over
      // thousands of tokens that shrinks it by 1e-5 and more.  So each step's
      // product starts afresh and is added with rounding.
      if constexpr (!Q4) {
        const uint32_t vbase = smem_addr(buf) + D / 64 * kTile * 128;
        const int tok = (lane & 7) + ((lane >> 4) << 3), ch = (lane >> 3) & 1;
        constexpr int JB = NT == 1 ? 4 : 2;  // independent products in flight: JB·NT
#pragma unroll
        for (int j0v = 0; j0v < MT; j0v += JB) {
          uint32_t af[JB][4];
          float t[JB][NT][4];
#pragma unroll
          for (int jj = 0; jj < JB; ++jj) {
            const int c = 2 * (j0v + jj) + ch;
            ldsm_x4_trans(vbase + (c >> 3) * (kTile * 128) + tok * 128 + (((c & 7) ^ (tok & 7)) << 4), af[jj]);
          }
#pragma unroll
          for (int part = 2; part >= 0; --part)
#pragma unroll
            for (int jj = 0; jj < JB; ++jj)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if (part == 2) mma_first(t[jj][nt], af[jj], pf[0][nt][part]);
                else mma(t[jj][nt], af[jj], pf[0][nt][part], t[jj][nt]);
              }
#pragma unroll
          for (int jj = 0; jj < JB; ++jj)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[j0v + jj][nt][e] += t[jj][nt][e];
        }
      } else {
        // The codes are numbers already, as K's.  To center them at 8, products with the first part of w start from −8·Σ hi,
        // computed by the same tensor cores from a tile of −8·2⁻¹³³, which loses
        // nothing, since hi has 8 bits; the other parts leave 8·Σ (mid + lo), small,
        // which corr takes back.  Codes in the upper places come 16 times too large;
        // their rows of the result are divided by 16 at the end.
        float c8[U][NT][2];
        const uint32_t m8[4] = {0x80088008u, 0x80088008u, 0x80088008u, 0x80088008u};
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float t[4];
            mma_first(t, m8, pf[u][nt][0]);
            c8[u][nt][0] = t[0];
            c8[u][nt][1] = t[1];
          }
        // lane (g, t4): tokens 2·t4, 2·t4 + 1 (+ 8), numbers D/8·g … of each;
        // the byte interleave pairs the two tokens' codes of one number
        constexpr int VW = D / 64;  // words per lane and token
        uint32_t un[U][2][2 * VW];  // [tokens, tokens + 8][four numbers each]
#pragma unroll
        for (int u = 0; u < U; ++u) {
          uint32_t wv[4][VW];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const unsigned char* src = buf + u * (Sh::slot_bytes / U) + 8 * D +
                                       (2 * t4 + (x & 1) + (x >> 1) * 8) * (D / 2) + g * (D / 16);
            if constexpr (VW == 2) {
              const uint2 y = *reinterpret_cast<const uint2*>(src);
              wv[x][0] = y.x;
              wv[x][1] = y.y;
            } else {
              wv[x][0] = *reinterpret_cast<const uint32_t*>(src);
            }
          }
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int w = 0; w < VW; ++w) {
              un[u][hf][2 * w] = __byte_perm(wv[2 * hf][w], wv[2 * hf + 1][w], 0x5410);
              un[u][hf][2 * w + 1] = __byte_perm(wv[2 * hf][w], wv[2 * hf + 1][w], 0x7632);
            }
        }
        // Rows in two sets, so that the four registers an offset needs are filled
        // once for each: even j (codes in the lower places), then odd j.
        constexpr int JB = 2;  // independent products in flight: U·JB·NT
#pragma unroll
        for (int odd = 0; odd < 2; ++odd) {
          float c[U][NT][4];
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) c[u][nt][e] = c8[u][nt][e & 1] * (odd ? 16.f : 1.f);
#pragma unroll
          for (int q = 0; q < MT / 2; q += JB) {
            uint32_t af[U][JB][4];
            float t[U][JB][NT][4];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int jj = 0; jj < JB; ++jj) {
                // m rows g: number j of the lane's share; rows g + 8: number MT + j
                const int j = 2 * (q + jj) + odd, sh = 8 * (j >> 1 & 1);
                const uint32_t mask = odd ? 0x00f000f0u : 0x000f000fu;
                af[u][jj][0] = (un[u][0][j / 4] >> sh) & mask;
                af[u][jj][1] = (un[u][0][MT / 4 + j / 4] >> sh) & mask;
                af[u][jj][2] = (un[u][1][j / 4] >> sh) & mask;
                af[u][jj][3] = (un[u][1][MT / 4 + j / 4] >> sh) & mask;
              }
#pragma unroll
            for (int part = 0; part < 3; ++part)
#pragma unroll
              for (int u = 0; u < U; ++u)
#pragma unroll
                for (int jj = 0; jj < JB; ++jj)
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt)
                    mma(t[u][jj][nt], af[u][jj], pf[u][nt][part], part == 0 ? c[u][nt] : t[u][jj][nt]);
#pragma unroll
            for (int jj = 0; jj < JB; ++jj)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  float sum = t[0][jj][nt][e];
                  if constexpr (U == 2) sum += t[U - 1][jj][nt][e];
                  o[2 * (q + jj) + odd][nt][e] += sum;
                }
          }
        }
      }
      // the slot is free: the next copies into it
      stream_sync();
      if (rg == 0 && lane / U == ((in + ST) & (kSteps - 1)) && k + ST < nk) {
        fence_proxy_async_shared();  // the slot's reads come before the copies that refill it
        issue(in + ST < kSteps ? cur : nxt, sl, lane % U);
      }
      if (++ring_at == ST) {
        ring_at = 0;
        parity ^= 1u;
      }
    }

    // ---- the next unit's copies start before this one's warps are added up
    bool more = false;
    if (!aligned) {
      pos += now.t1 - now.t0;
      more = pos < end;
      if (more) {
        if (pos >= grp_at + static_cast<long long>(seg.n) * mult) {
          grp_at += static_cast<long long>(seg.n) * mult;
          ++grp;
          seg.n = group_tiles(a, grp);
          seg.vis = visible_tiles(a, load_bounds(a, a.sel ? grp / a.Hkv : grp));
        }
        place();
        prologue(seg, true);
        if (tid == 0) s_seg[which ^ 1] = seg;
      }
    }

#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) {
          l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], sh);
          if constexpr (Q4) corr[nt][e] += __shfl_xor_sync(0xffffffffu, corr[nt][e], sh);
        }
        if (g == 0) {
          s_m[warp][nt * 8 + 2 * t4 + e] = m[nt][e] == kNoMax ? -INFINITY : m[nt][e];
          s_l[warp][nt * 8 + 2 * t4 + e] = l[nt][e];
          s_c[warp][nt * 8 + 2 * t4 + e] = corr[nt][e];
        }
      }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = nt * 8 + 2 * t4 + e;
        float top = -INFINITY;
#pragma unroll
        for (int s = 0; s < NS; ++s) top = fmaxf(top, s_m[s * R + rg][row]);
        const float mine = s_m[warp][row], f = mine > -INFINITY ? ex2(mine - top) : 0.f;
        float* to = red + (warp * 8 * NT + row) * PITCH;
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          // 4 bits: back from 2^(64 − 133), and from 16 times that for odd j
          const float by = Q4 ? f * (j & 1 ? 0x1p65f : 0x1p69f) : f;
          to[merge_at<D, Q4>(Q4 ? D / 8 * g + j : 16 * j + g)] = o[j][nt][e] * by;
          to[merge_at<D, Q4>(Q4 ? D / 8 * g + MT + j : 16 * j + 8 + g)] = o[j][nt][2 + e] * by;
        }
      }
    const bool entire = now.t0 == 0 && now.t1 == now.n;
    const int slot = 2 * blockIdx.x + (first_segment ? 0 : 1);
    if (tid < rows) {  // one thread per row: its maximum and sum, and where they go
      const int r = tid / (8 * NT), in = tid - r * (8 * NT);
      float top = -INFINITY, den = 0.f, cc = 0.f;
#pragma unroll
      for (int s = 0; s < NS; ++s) top = fmaxf(top, s_m[s * R + r][in]);
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int w = s * R + r;
        const float f = s_m[w][in] > -INFINITY ? ex2(s_m[w][in] - top) : 0.f;
        den = fmaf(s_l[w][in], f, den);
        cc = fmaf(s_c[w][in], f, cc);
      }
      if (entire) {
        const bool none = top == -INFINITY && den == den;  // no visible token with a score above −inf
        s_row[tid] = make_float2(none ? 0.f : 1.f / den, cc);
        if (a.lse) {
          const int t = tid >> a.gsh, hq = now.h * a.G + tid - (t << a.gsh);
          float lse = none ? -INFINITY : (top + log2f(den)) * kLn2;
          if (a.slopes && !none) {
            const float sl = a.slopes[hq];
            lse -= sl * static_cast<float>(ref_distance(sl, now.vis.L - a.T + t, ref));
          }
          a.lse[(static_cast<size_t>(now.b) * a.T + t) * a.Hq + hq] = lse;
        }
      } else {
        s_row[tid] = make_float2(1.f, cc);
        a.ml[static_cast<size_t>(slot) * rows + tid] = make_float2(top, den);
      }
    }
    __syncthreads();
#pragma unroll 2
    for (int i = tid; i < rows * (D / 4); i += Sh::threads) {
      const int row = i / (D / 4), c = (i - row * (D / 4)) * 4, r = row / (8 * NT), in = row - r * (8 * NT);
      const float2 by = s_row[row];
      float4 sum = Q4 ? make_float4(by.y, by.y, by.y, by.y) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const float* from = red + ((s * R + r) * 8 * NT + in) * PITCH + merge_at<D, Q4>(c);
        const float4 x = Q4 ? make_float4(from[0], from[1], from[2], from[3]) : *reinterpret_cast<const float4*>(from);
        sum.x += x.x;
        sum.y += x.y;
        sum.z += x.z;
        sum.w += x.w;
      }
      const int t = row >> a.gsh, hq = now.h * a.G + row - (t << a.gsh);
      float* to = entire ? a.out + ((static_cast<size_t>(now.b) * a.T + t) * a.Hq + hq) * D + c
                         : a.part + (static_cast<size_t>(slot) * rows + row) * D + c;
      *reinterpret_cast<float4*>(to) = make_float4(sum.x * by.x, sum.y * by.x, sum.z * by.x, sum.w * by.x);
    }
    if (!entire && tid == 0) {
      a.ref[slot] = ref;
      // the unit's first piece: the CTAs that follow hold the others
      if (now.t0 == 0) a.cut[blockIdx.x] = make_int4(now.unit, slot, now.pieces, 0);
    }
    if (!more) return;
    first_segment = false;
    __syncthreads();
    which ^= 1;
  }
}

// grid (CTAs of mod_kernel, blocks of kMerge/(D/4) rows): adds the pieces of the
// unit that CTA x cut, in CTA order.  A thread takes four numbers of a row over
// every slices-th piece (one slice where the rows fill the block), eight pieces'
// loads at a time: the chain of dependent loads is what bounds it, and one block
// per CTA for up to 16 rows keeps it to one wave.
constexpr int kMerge = 512;
template <int D>
__global__ void __launch_bounds__(kMerge) mod_combine_kernel(ModArgs a) {
  grid_dep_enter();
  const int4 cut = a.cut[blockIdx.x];
  if (cut.z <= 1) return;
  constexpr int kAhead = 8;
  __shared__ float4 s_num[kMerge];
  __shared__ float2 s_ml[kMerge];
  const int rows = a.G * a.T, items = rows * (D / 4);
  const int slices = items < kMerge ? kMerge / items : 1;
  const int sl = items < kMerge ? static_cast<int>(threadIdx.x) / items : 0;
  const int item = blockIdx.y * kMerge + threadIdx.x - sl * items;
  const bool live = sl < slices && item < items;
  const int row = live ? item / (D / 4) : 0, c = (item % (D / 4)) * 4, cta = blockIdx.x, n = cut.z;
  const int b = cut.x / a.Hkv, h = cut.x - b * a.Hkv, t = row >> a.gsh, hq = h * a.G + row - (t << a.gsh);
  auto slot = [&](int p) { return static_cast<size_t>(p == 0 ? cut.y : 2 * (cta + p)); };
  float slope = 0.f;
  int qpos = 0, base = 0;
  if (a.slopes) {
    slope = a.slopes[hq];
    const int L = a.seq_lens[b], most = a.max_pages * a.S;
    qpos = (L < 0 ? 0 : (L > most ? most : L)) - a.T + t;
    // the pieces' biases are measured from distances of their own: all to the
    // last piece's (the nearest tokens), or the first's for a rising bias
    base = ref_distance(slope, qpos, a.ref[slot(slope >= 0.f ? n - 1 : 0)]);
  }
  float m = -INFINITY, den = 0.f;
  float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float m2, float den2, float4 x) {
    const float up = fmaxf(m, m2);
    const float f = m > -INFINITY ? ex2(m - up) : 0.f, f2 = m2 > -INFINITY ? ex2(m2 - up) : 0.f;
    den = den * f + den2 * f2;
    num = make_float4(fmaf(num.x, f, x.x * f2), fmaf(num.y, f, x.y * f2), fmaf(num.z, f, x.z * f2),
                      fmaf(num.w, f, x.w * f2));
    m = up;
  };
  if (live) {
    for (int p0 = sl; p0 < n; p0 += kAhead * slices) {
      float4 x[kAhead];
      float2 ml[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const size_t at = slot(min(p0 + i * slices, n - 1)) * rows + row;
        x[i] = *reinterpret_cast<const float4*>(a.part + at * D + c);
        ml[i] = a.ml[at];
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int p = p0 + i * slices;
        if (p >= n) break;
        float top = ml[i].x;
        if (a.slopes) top -= slope * kLog2e * static_cast<float>(ref_distance(slope, qpos, a.ref[slot(p)]) - base);
        add(top, ml[i].y, x[i]);
      }
    }
  }
  if (slices > 1) {
    s_num[threadIdx.x] = num;
    s_ml[threadIdx.x] = make_float2(m, den);
    __syncthreads();
    if (sl != 0) return;
    for (int k = 1; k < slices; ++k) {
      const float2 ml = s_ml[threadIdx.x + k * items];
      add(ml.x, ml.y, s_num[threadIdx.x + k * items]);
    }
  }
  if (!live) return;
  const size_t orow = (static_cast<size_t>(b) * a.T + t) * a.Hq + hq;
  const bool none = m == -INFINITY && den == den;
  const float by = 1.f / den;
  *reinterpret_cast<float4*>(a.out + orow * D + c) =
      none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(num.x * by, num.y * by, num.z * by, num.w * by);
  if (c == 0 && a.lse) a.lse[orow] = none ? -INFINITY : (m + log2f(den)) * kLn2 - slope * static_cast<float>(base);
}

// Two-dimensional view [rows, d] of a pool, copied 16 rows × 64 columns at a
// time with the 128-byte swizzle, which keeps the fragment loads of both
// products free of bank conflicts.
cudaError_t pool_map(CUtensorMap* map, void* pool, size_t rows, int d) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static Encode encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r);
    return e == cudaSuccess && r == cudaDriverEntryPointSuccess ? reinterpret_cast<Encode>(f) : nullptr;
  }();
  if (encode == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dim[2] = {static_cast<cuuint64_t>(d), rows}, stride[1] = {static_cast<cuuint64_t>(d) * 2};
  const cuuint32_t box[2] = {64, kTile}, one[2] = {1, 1};
  const CUresult r =
      encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, pool, dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

inline size_t al256(size_t x) { return (x + 255) / 256 * 256; }

template <int D, int NT, int R, bool Q4>
cudaError_t run_mod(const ModArgs& a, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t st) {
  constexpr size_t smem = mod_smem<D, NT, R, Q4>();
  static std::atomic<uint64_t> ready{0};  // devices on which the kernel may have that much shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev >= 64 || !(ready.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(mod_kernel<D, NT, R, Q4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  const int ctas = min(kModCtas, 2 * sm_count());
  e = launch_k(mod_kernel<D, NT, R, Q4>, dim3(static_cast<unsigned>(ctas)), Shape<D, NT, Q4>::threads, smem, st, km, vm, a);
  if (e != cudaSuccess) return e;
  const int items = a.G * a.T * (D / 4);
  return launch_k(mod_combine_kernel<D>, dim3(static_cast<unsigned>(ctas), static_cast<unsigned>((items + kMerge - 1) / kMerge)),
                  kMerge, 0, st, a);
}

template <int D, bool Q4>
cudaError_t dispatch_rows(const ModArgs& a, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t st) {
  const int rows = a.G * a.T;
  if (rows <= 8) return run_mod<D, 1, 1, Q4>(a, km, vm, st);
  if (rows <= 16) return run_mod<D, 2, 1, Q4>(a, km, vm, st);
  if (rows <= 32) return run_mod<D, 2, 2, Q4>(a, km, vm, st);
  return run_mod<D, 2, 4, Q4>(a, km, vm, st);
}

}  // namespace

size_t softmax_mod_ws_bytes(int d, int rows) {
  const size_t slots = 2 * static_cast<size_t>(kModCtas);
  return al256(slots * rows * d * sizeof(float)) + al256(slots * rows * sizeof(float2)) + al256(slots * sizeof(int2)) +
         al256(kModCtas * sizeof(int4));
}

// pool: the 4-bit pool, or NULL for the bf16 pools of c.
cudaError_t launch_softmax_mod(const ekv_cache& c, const void* pool, const ekv_seqs& s, const void* q, int Hq, int T,
                               float scale, const ekv_score_mod* mod, const int32_t* sel, const int32_t* n_sel,
                               int cap, float* out, float* lse, void* ws, cudaStream_t st) {
  ModArgs a{};
  a.page_table = s.page_table;
  a.seq_lens = s.seq_lens;
  a.q = static_cast<const bf16*>(q);
  a.sel = sel;
  a.n_sel = n_sel;
  a.pool = static_cast<const unsigned char*>(pool);
  a.out = out;
  a.lse = lse;
  a.batch = s.batch;
  a.Hkv = c.num_kv_heads;
  a.Hq = Hq;
  a.G = Hq / c.num_kv_heads;
  while ((1 << a.gsh) < a.G) ++a.gsh;
  a.T = T;
  a.S = c.page_size;
  a.num_phys = c.num_phys_pages;
  a.max_pages = s.max_pages;
  a.cap = cap;
  a.min_tiles = pool ? 8 : 4;
  a.slack_tiles = pool ? 32 : 12;
  auto finite = [](float x) { return x < kHuge ? x : kHuge; };  // so that a sum of 0 stays 0
  a.scale2 = finite(scale * kLog2e);
  if (mod != nullptr) {
    a.slopes = mod->slopes;
    a.prefix_lens = mod->prefix_lens;
    a.starts = mod->starts;
    a.window = mod->window;
    // a cap of 1e30 changes no score in fp32; under 1e-30 scores are ±cap or 0
    if (mod->softcap > 0.f && mod->softcap < 1e30f) {
      a.capx = finite(scale / fmaxf(mod->softcap, 1e-30f));
      a.cap2 = mod->softcap * kLog2e;
    }
  }
  const int d = c.head_dim, rows = a.G * T;
  const size_t slots = 2 * static_cast<size_t>(kModCtas);
  char* p = static_cast<char*>(ws);
  a.part = reinterpret_cast<float*>(p);
  p += al256(slots * rows * d * sizeof(float));
  a.ml = reinterpret_cast<float2*>(p);
  p += al256(slots * rows * sizeof(float2));
  a.ref = reinterpret_cast<int2*>(p);
  p += al256(slots * sizeof(int2));
  a.cut = reinterpret_cast<int4*>(p);
  CUtensorMap km{}, vm{};
  if (pool == nullptr) {
    const size_t pool_rows = static_cast<size_t>(c.num_phys_pages) * c.num_kv_heads * c.page_size;
    cudaError_t e = pool_map(&km, c.k_pool, pool_rows, d);
    if (e == cudaSuccess) e = pool_map(&vm, c.v_pool, pool_rows, d);
    if (e != cudaSuccess) return e;
    return d == 128 ? dispatch_rows<128, false>(a, km, vm, st) : dispatch_rows<64, false>(a, km, vm, st);
  }
  return d == 128 ? dispatch_rows<128, true>(a, km, vm, st) : dispatch_rows<64, true>(a, km, vm, st);
}

}  // namespace ekv
