// attention_kernel.cuh — attention of new tokens over the 8-bit paged cache
// (spec_attention).
//
// For one request and key head, the rows of Q are its new tokens times the
// query heads of the group.  Positions go in tiles of 128:
//
//   S^T [128 positions x rows]  = K [positions x D] Q^T         (K: A operand)
//   O^T [D x rows]             += V^T [D x positions] P^T       (V: A operand)
//
// Positions are the M of the first product and D the M of the second, so that
// few rows cost little (they are the N), and a thread's values all belong to
// one position: its scales are two numbers.
//
// First product: e4m3 x e4m3 with 32-bit sums.  K goes from HBM to the tensor
// cores as it lies in the cache.  Q, bf16 scaled by a power of two a row, is
// the sum of two e4m3 numbers: a value of 8 significant bits is its nearest
// number of 4 bits plus a remainder of 4 (exact to 2^-18 of the row's largest).
//
// Second product: f16 x f16.  An e4m3 V is exact in f16, and one group of
// warps turns V's tiles over while the softmax is at work; P in f16 has 11
// bits down to 2^-20 of its reference and 2^-31 of it is lost.  (P as two e4m3
// numbers needs no such step, but loses what is below 2^-22 of the largest,
// which a faint tail after one strong position is, and costs twice the
// arithmetic a probability.)
//
// The reference of a row is its largest score when it was last looked for: in
// the first tile, and whenever a later score lies more than 2^9 above it.  So
// O stays in tensor memory, and most tiles need no search for a maximum.
//
// Two groups of four warps do the softmax.  Up to 32 rows each takes every
// other tile, with references, sums and an O of its own, which the output
// warps add up: a tile then has the time of two.  Above 32 rows each takes
// half of the rows of every tile, so that a thread's scores and sums stay in
// registers.
//
// The tiles of all requests, heads and row groups form one list that is cut
// into equal parts, one for each CTA; what a cut separates is joined by the
// CTA that finishes last, in the order of the parts.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "kv_kernels.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace specdec {

struct AttnArgs {
  const __nv_bfloat16* q;
  long long q_stride;  // elements
  __nv_bfloat16* out;
  int32_t T, Hq, H, B;
  const int32_t* cu_tokens;
  const int32_t* kv_len;
  const int32_t* table;
  int32_t max_blocks, num_blocks, bs, bs_log2;
  const float* k_scale;
  const float* v_scale;
  float scale_log2e;
  uint32_t* err;
  uint32_t* counters;  // one for each CTA, zero between calls
  float* partial;      // two records for each CTA
  int32_t ring;        // tiles of K, and of V, in shared memory
  int32_t rows;        // most rows of a tile, a multiple of 16
};

constexpr int kTile = 128;      // positions of a tile
constexpr int kAttnRows = 64;   // most rows of a tile
constexpr int kHalfRows = kAttnRows / 2;  // most of a softmax group
// Warps: 0-3 and 4-7 softmax, 8-11 V to f16, 12-15 Q and O, 16 copies, 17 first
// products, 18 second products, 19 the list of segments.
constexpr int kAttnThreads = 640;
// Registers a thread: 96 at launch, moved to the softmax, whose scores and
// sums are 64 of them.
constexpr int kRegsSoftmax = 120, kRegsValues = 72, kRegsOutput = 96, kRegsRest = 64;
static_assert(256 * kRegsSoftmax + 128 * (kRegsValues + kRegsOutput + kRegsRest) <= 96 * kAttnThreads,
              "the warpgroups' registers are those of the launch");
constexpr int kScaleRing = 8;
constexpr int kSegRing = 4;
constexpr int kMaxRing = 8;     // tiles of K, and of V, in shared memory
constexpr int kMaxPages = 8;    // blocks of a tile
constexpr uint32_t kTmemCols = 256;  // S twice, O twice
constexpr int kPartialFloats = kAttnRows * 128 + 2 * kAttnRows;
// P = 2^kPScale at the reference score; a score may pass it by 2^kSlack
// before P would leave f16.
constexpr float kPScale = 64.f;
constexpr float kSlack = 9.f;
// A wait gives up after this many tries of at most a microsecond each.
#ifndef SPECDEC_ATTN_WAIT_TRIES
#define SPECDEC_ATTN_WAIT_TRIES 2000000u
#endif

// Part of a (request, head, row group) that one CTA works on.  tile1 < 0 ends
// the list.
struct Segment {
  int b, h, row0, rows;       // rows of this group
  int q0, kv, len;            // first token, positions before it, positions of the group
  int tile0, tile1, tiles;    // tiles of this part, and of the whole
  long long first;            // unit of the whole's first tile
};

// Goes through the segments of units [u, end).
struct Walker {
  const AttnArgs& a;
  long long u, end, ub;  // ub: first unit of request b
  int b, G, q0, q, kv;
  long long per_head;

  __device__ Walker(const AttnArgs& args, long long u0, long long u1, int b0, long long ub0)
      : a(args), u(u0), end(u1), ub(ub0), b(b0), G(args.Hq / args.H) {
    if (u < end) load();
  }
  // positions of the row group that ends before row `last`
  static __device__ int length(const AttnArgs& a, int kv, int G, int row_end) {
    const long long n = static_cast<long long>(kv) + (row_end - 1) / G + 1;
    const long long cap = static_cast<long long>(a.max_blocks) * a.bs;
    return static_cast<int>(n < 0 ? 0 : (n < cap ? n : cap));
  }
  static __device__ int tiles_of(int len) { return len <= 0 ? 1 : (len + kTile - 1) / kTile; }
  static __device__ long long units_per_head(const AttnArgs& a, int kv, int G, int q) {
    long long n = 0;
    for (int r = 0; r < q * G; r += a.rows) n += tiles_of(length(a, kv, G, min(q * G, r + a.rows)));
    return n;
  }
  static __device__ void request(const AttnArgs& a, int b, int& q0, int& q, int& kv) {
    q0 = max(0, min(__ldg(a.cu_tokens + b), a.T));
    const int q1 = max(0, min(__ldg(a.cu_tokens + b + 1), a.T));
    q = max(0, q1 - q0);
    kv = __ldg(a.kv_len + b);
  }
  __device__ void load() {
    request(a, b, q0, q, kv);
    per_head = units_per_head(a, kv, G, q);
  }
  __device__ bool next(Segment& s) {
    if (u >= end) return false;
    while (u >= ub + per_head * a.H) {
      ub += per_head * a.H;
      ++b;
      load();
    }
    const long long o = u - ub;
    s.b = b;
    s.h = static_cast<int>(o / per_head);
    long long rem = o - s.h * per_head;
    s.q0 = q0;
    s.kv = kv;
    for (s.row0 = 0;; s.row0 += a.rows) {
      const int row_end = min(q * G, s.row0 + a.rows);
      s.rows = row_end - s.row0;
      s.len = length(a, kv, G, row_end);
      s.tiles = tiles_of(s.len);
      if (rem < s.tiles) break;
      rem -= s.tiles;
    }
    s.tile0 = static_cast<int>(rem);
    s.tile1 = static_cast<int>(min(static_cast<long long>(s.tiles), rem + (end - u)));
    s.first = u - rem;
    u += s.tile1 - s.tile0;
    return true;
  }
};

struct ScaleEntry {
  float ks[kMaxPages];   // key scale times the scores' factor
  float vs[kMaxPages];   // value scale
  float vmax;            // the tile's largest
};

struct AttnShared {
  uint64_t k_full[kMaxRing], k_empty[kMaxRing], v_full[kMaxRing], v_empty[kMaxRing];
  uint64_t s_full[2], s_empty[2], p_full[2], f_full[2], pv_done[2], o_full[2], o_empty[2];
  uint64_t q_full, q_empty, meta_full[2], l_full[2];
  uint64_t sc_full[kScaleRing], sc_empty[kScaleRing], seg_full[kSegRing], seg_empty[kSegRing], done[2];
  uint32_t tmem;
  int32_t b0;
  long long ub0;
  Segment seg[kSegRing];
  long long part[32];
  alignas(16) float2 col[2][kHalfRows];  // {row scale, reference} of each group's rows
  float wmax[2][4][kHalfRows];        // a warp's largest score of each of its group's rows
  float fac[2][kHalfRows];            // factors from a row's reference to its next
  float qs[2][kAttnRows];
  int32_t limit[2][kAttnRows];        // last position a row attends to
  float lsum[2][8][kHalfRows];        // sums of the softmax warps
  float mrun[2][2][kHalfRows];        // and their groups' references
  float vref[2][2];
  alignas(16) float4 fin[kAttnRows];  // {factor of one group's O, of the other's, sum (or its inverse), reference}
  int32_t nanpos[2][128];             // first new position whose value is NaN in a dimension
  ScaleEntry scales[kScaleRing];
  int32_t last;
};

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Whether `x` holds for any thread of the barrier.
__device__ __forceinline__ bool named_any(int id, int threads, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

// A wait that gives up once; after that the thread goes on without waiting, so
// that every barrier still gets its arrivals, to the end of its segment.  What
// decides how often a group of warps meets at a barrier is agreed on at one.
struct Waiter {
  bool dead = false;
  __device__ __forceinline__ void operator()(const uint64_t& bar, uint32_t parity) {
    if (dead) return;
    const uint32_t at = ptx::smem_addr(&bar);
    for (uint32_t n = SPECDEC_ATTN_WAIT_TRIES; !tc::try_wait(at, parity);)
      if (--n == 0) {
        dead = true;
        break;
      }
  }
};
// Arrivals for the warp, after what all its threads did before.
__device__ __forceinline__ void warp_arrive(uint64_t& bar, uint32_t n = 1) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0)
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(ptx::smem_addr(&bar)), "r"(n) : "memory");
}

// Nearest number of 4 significant bits; the remainder of a number of 8 has 4.
__device__ __forceinline__ float top4(float x) {
  return __uint_as_float((__float_as_uint(x) + 0x80000u) & 0xFFF00000u);
}

// Byte x of row t in a tile of K or V (rows of D bytes) as the copies swizzle it.
template <int D>
__device__ __forceinline__ int swizzled(int t, int x) {
  return D == 128 ? t * 128 + (x ^ ((t & 7) << 4)) : t * 64 + (x ^ (((t >> 1) & 3) << 4));
}

// Sums of 8 values over the warp: lane i gets that of value i >> 2.
__device__ __forceinline__ float warp_sums8(const float* v) {
  const int lane = threadIdx.x & 31;
  float a[4], b[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool up = lane & 16;
    a[i] = (up ? v[i + 4] : v[i]) + __shfl_xor_sync(0xFFFFFFFFu, up ? v[i] : v[i + 4], 16);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool up = lane & 8;
    b[i] = (up ? a[i + 2] : a[i]) + __shfl_xor_sync(0xFFFFFFFFu, up ? a[i] : a[i + 2], 8);
  }
  const bool up = lane & 4;
  float s = (up ? b[1] : b[0]) + __shfl_xor_sync(0xFFFFFFFFu, up ? b[0] : b[1], 4);
  s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
  return s + __shfl_xor_sync(0xFFFFFFFFu, s, 1);
}

template <int D>
struct AttnLayout {
  static constexpr int kTileBytes = kTile * D;       // of K or V
  static constexpr int kHalfBytes = kTile * D * 2;   // of V in f16
  static __host__ __device__ int q_bytes(int rows) { return rows * D; }          // of one half
  static __host__ __device__ int p_bytes(int rows) { return rows * kTile * 2; }  // of one buffer
  static __host__ __device__ int tiles_at() { return (static_cast<int>(sizeof(AttnShared)) + 1023) / 1024 * 1024; }
  static __host__ __device__ int bytes(int ring, int rows) {
    return 1024 + tiles_at() + 2 * ring * kTileBytes + 2 * kHalfBytes + 2 * q_bytes(rows) + 2 * p_bytes(rows);
  }
};

template <int D>
__global__ void __launch_bounds__(kAttnThreads, 1)
    attention_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
  using L = AttnLayout<D>;
  extern __shared__ __align__(16) unsigned char raw[];
  unsigned char* base = raw + ((1024u - (ptx::smem_addr(raw) & 1023u)) & 1023u);
  AttnShared& sh = *reinterpret_cast<AttnShared*>(base);
  unsigned char* k_tiles = base + L::tiles_at();
  unsigned char* v_tiles = k_tiles + a.ring * L::kTileBytes;
  unsigned char* v_half = v_tiles + a.ring * L::kTileBytes;
  unsigned char* q_hi = v_half + 2 * L::kHalfBytes;
  unsigned char* q_lo = q_hi + L::q_bytes(a.rows);
  unsigned char* p_at = q_lo + L::q_bytes(a.rows);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = a.Hq / a.H;

  if (tid == 0) {
    auto init = [](uint64_t& bar, uint32_t n) { ptx::mbar_init(ptx::smem_addr(&bar), n); };
    for (int i = 0; i < a.ring; ++i) {
      init(sh.k_full[i], 1);
      init(sh.k_empty[i], 1);
      init(sh.v_full[i], 1);
      init(sh.v_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      init(sh.s_full[i], 1);
      init(sh.s_empty[i], 8);
      init(sh.p_full[i], 8);
      init(sh.f_full[i], 4);
      init(sh.pv_done[i], 1);
      init(sh.o_full[i], 1);
      init(sh.o_empty[i], 4);
      init(sh.meta_full[i], 4);
      init(sh.l_full[i], 12);
    }
    for (int i = 0; i < kScaleRing; ++i) {
      init(sh.sc_full[i], 1);
      init(sh.sc_empty[i], 8);
    }
    init(sh.q_full, 4);
    init(sh.q_empty, 1);
    init(sh.done[0], 1);
    init(sh.done[1], 1);
    for (int i = 0; i < kSegRing; ++i) {
      init(sh.seg_full[i], 1);
      init(sh.seg_empty[i], 19);
    }
    ptx::fence_mbarrier_init();
    sh.b0 = 0;
    sh.ub0 = 0;
  }
  if (warp == 17) tc::alloc(ptx::smem_addr(&sh.tmem), kTmemCols);

  // Units of all requests, and where this CTA's begin.
  long long u0, u1, chunk;
  {
    const int per = (a.B + kAttnThreads - 1) / kAttnThreads;
    const int lo = min(a.B, tid * per), hi = min(a.B, lo + per);
    long long mine = 0;
    for (int b = lo; b < hi; ++b) {
      int q0, q, kv;
      Walker::request(a, b, q0, q, kv);
      mine += Walker::units_per_head(a, kv, G, q) * a.H;
    }
    long long s = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xFFFFFFFFu, s, d);
      if (lane >= d) s += o;
    }
    if (lane == 31) sh.part[warp] = s;
    __syncthreads();
    long long before = s - mine, total = 0;
    for (int w = 0; w < kAttnThreads / 32; ++w) {
      if (w < warp) before += sh.part[w];
      total += sh.part[w];
    }
    chunk = (total + gridDim.x - 1) / gridDim.x;
    u0 = min(total, static_cast<long long>(blockIdx.x) * chunk);
    u1 = min(total, u0 + chunk);
    if (u0 < u1 && before <= u0 && u0 < before + mine) {  // one thread
      long long at = before;
      for (int b = lo; b < hi; ++b) {
        int q0, q, kv;
        Walker::request(a, b, q0, q, kv);
        const long long n = Walker::units_per_head(a, kv, G, q) * a.H;
        if (u0 < at + n) {
          sh.b0 = b;
          sh.ub0 = at;
          break;
        }
        at += n;
      }
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
  }
  const uint32_t tmem = sh.tmem;
  Waiter wait;
  // The n-th segment, or null at the list's end; and the warp is done with it.
  auto segment = [&](int n) -> const Segment* {
    wait(sh.seg_full[n % kSegRing], (n / kSegRing) & 1);
    wait.dead = __any_sync(0xFFFFFFFFu, wait.dead);
    const Segment* s = &sh.seg[n % kSegRing];
    return wait.dead || s->tile1 < 0 ? nullptr : s;
  };
  auto leave = [&](int n) { warp_arrive(sh.seg_empty[n % kSegRing]); };

  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    // A thread has one position and the rows of its group.
    tc::more_registers<kRegsSoftmax>();
    const int grp = warp >> 2, t_in = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int page = t_in >> a.bs_log2;
    float x[kHalfRows], l[kHalfRows];
    const float4* col = reinterpret_cast<const float4*>(sh.col[grp]);
    int k0 = 0;  // tiles of the segments before
    for (int n_seg = 0;; ++n_seg) {
      const Segment* seg = segment(n_seg);
      // (and the last segment's rows are no longer read)
      if (named_any(1 + grp, 128, seg == nullptr)) break;
      const int par = n_seg & 1;
      const bool by_rows = seg->rows > kHalfRows;
      const int step = by_rows ? 1 : 2;
      // groups of 8 rows, and the first row
      const int eights = by_rows ? (seg->rows + 15) / 16 : (seg->rows + 15) / 16 * 2;
      const int r0 = by_rows ? grp * eights * 8 : 0;
      const int tiles = seg->tile1 - seg->tile0, len = seg->len;
      const int all_see = seg->kv + seg->row0 / G;  // last position that all rows attend to
      int pos0 = seg->tile0 * kTile;
      const uint32_t o_at = tmem + lanes + (2 + par) * kAttnRows + (by_rows ? r0 : grp * kHalfRows);
      float vref = 1.f, vinv = 1.f;
#pragma unroll
      for (int r = 0; r < kHalfRows; ++r) l[r] = 0.f;
      wait(sh.meta_full[par], (n_seg >> 1) & 1);
      if (t_in < eights * 8) sh.col[grp][t_in] = make_float2(sh.qs[par][r0 + t_in], 0.f);
      named_barrier(1 + grp, 128);
      bool first = true;
      // by tiles: those whose number is of the group's parity
      int i = by_rows ? 0 : ((k0 ^ grp) & 1);
      pos0 += i * kTile;
      for (; i < tiles; i += step, pos0 += step * kTile) {
        const int k = k0 + i, pos = pos0 + t_in;
        const bool masked = pos0 + kTile - 1 > all_see || pos0 + kTile > len;
        const ScaleEntry& sc = sh.scales[k % kScaleRing];
        wait(sh.sc_full[k % kScaleRing], (k / kScaleRing) & 1);
        const float ks = sc.ks[page], vs = sc.vs[page], vmax = sc.vmax;
        warp_arrive(sh.sc_empty[k % kScaleRing], step);
        bool renew = first;
        wait(sh.s_full[k & 1], (k >> 1) & 1);
        tc::fence_after();
        const uint32_t s_at = tmem + lanes + (k & 1) * kAttnRows + r0;
        for (;;) {
          if (renew) {
            // New references: the rows' largest scores so far, and the largest
            // value scale where it has grown.
            const float vref_was = vref;
            if (first || vmax > 4.f * vref) {
              vref = vmax > 0x1p-100f ? vmax : 0x1p-100f;
              vinv = 1.f / vref;
            }
#pragma unroll 1
            for (int c = 0; c < eights; ++c) {
              float v[8], mine = -INFINITY;
              tc::ld8(s_at + c * 8, v);
              tc::wait_ld();
              tc::ready(v);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                float y = v[e] * ks * sh.col[grp][c * 8 + e].x;
                if (masked && pos > sh.limit[par][r0 + c * 8 + e]) y = -INFINITY;
                y = tc::warp_max(y);
                if (lane == e) mine = y;
              }
              if (lane < 8) sh.wmax[grp][warp & 3][c * 8 + lane] = mine;
            }
            if (!first) wait(sh.pv_done[(k - step) & 1], ((k - step) >> 1) & 1);  // O rests
            tc::fence_after();
            named_barrier(1 + grp, 128);
            if (t_in < eights * 8) {
              const float m = fmaxf(fmaxf(sh.wmax[grp][0][t_in], sh.wmax[grp][1][t_in]),
                                    fmaxf(sh.wmax[grp][2][t_in], sh.wmax[grp][3][t_in]));
              const float was = sh.col[grp][t_in].y;
              const float now = first ? (m > -INFINITY ? m : 0.f) : fmaxf(was, m);
              sh.col[grp][t_in].y = now;
              sh.fac[grp][t_in] = tc::ex2(was - now);
            }
            named_barrier(1 + grp, 128);
            if (!first) {
#pragma unroll
              for (int r = 0; r < kHalfRows; ++r)
                if (r < eights * 8) l[r] *= sh.fac[grp][r];
              const float v_ratio = vref_was * vinv;
#pragma unroll 1
              for (int c = 0; c < eights; ++c) {
                float o[8];
                tc::ld8(o_at + c * 8, o);
                tc::wait_ld();
                tc::ready(o);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] *= sh.fac[grp][c * 8 + e] * v_ratio;
                tc::st8(o_at + c * 8, o);
              }
              tc::wait_st();
              tc::fence_before();
            }
          }
          // scores over the rows' references
#pragma unroll
          for (int c = 0; c < kHalfRows / 8; ++c)
            if (c < eights) tc::ld8(s_at + c * 8, x + c * 8);
          tc::wait_ld();
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < kHalfRows / 8; ++c) {
            if (c >= eights) break;
            tc::ready(x + c * 8);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const int r = c * 8 + e;
              const float4 w = col[r >> 1];
              x[r] = fmaf(x[r] * ks, w.x, -w.y);
              x[r + 1] = fmaf(x[r + 1] * ks, w.z, -w.w);
            }
            if (masked) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (pos > sh.limit[par][r0 + c * 8 + e]) x[c * 8 + e] = -INFINITY;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, x[c * 8 + e]);
          }
          // does P stay within f16 (and the sum within 32 bits)?
          if (renew || !named_any(1 + grp, 128, top > fminf(kSlack - __log2f(vs * vinv), 60.f) || vmax > 4.f * vref)) break;
          renew = true;
        }
        const float vr = vs * vinv * kPScale;
        tc::fence_before();
        warp_arrive(sh.s_empty[k & 1], step);
        first = false;
        if (k >= 2) wait(sh.pv_done[k & 1], ((k >> 1) - 1) & 1);
        // probabilities
        unsigned char* p = p_at + (k & 1) * L::p_bytes(a.rows) + (r0 / 8) * (16 * kTile) + t_in * 16;
#pragma unroll
        for (int c = 0; c < kHalfRows / 8; ++c) {
          if (c >= eights) break;
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const int r = c * 8 + e;
            const float p0 = tc::ex2(x[r]), p1 = tc::ex2(x[r + 1]);
            l[r] += p0;
            l[r + 1] += p1;
            w[e >> 1] = tc::f16x2(p0 * vr, p1 * vr);
          }
          *reinterpret_cast<uint4*>(p + c * (16 * kTile)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        tc::fence_smem();
        warp_arrive(sh.p_full[k & 1], step);
      }
      k0 += tiles;
      // sums and references for the output warps
#pragma unroll
      for (int c = 0; c < kHalfRows / 8; ++c) {
        if (c >= eights) break;
        const float s = warp_sums8(l + c * 8);
        if ((lane & 3) == 0) sh.lsum[par][warp][c * 8 + (lane >> 2)] = s;
      }
      if (t_in < eights * 8) sh.mrun[par][grp][t_in] = sh.col[grp][t_in].y;
      if (t_in == 0) sh.vref[par][grp] = vref / kPScale;
      warp_arrive(sh.l_full[par]);
      leave(n_seg);
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ V to f16
    // A thread has one position.  Values past the last position are no numbers
    // of the request's: zeros.  New positions are not seen by all rows: their
    // NaN leave the product, where 0 times NaN would spoil rows that do not
    // see them, and are noted for the output.
    tc::fewer_registers<kRegsValues>();
    const int t_in = tid - 256;
    int k = 0, slot = 0, round = 0;
    for (int n_seg = 0;; ++n_seg) {
      const Segment* seg = segment(n_seg);
      if (seg == nullptr) break;
      const int par = n_seg & 1, tile1 = seg->tile1, kv = seg->kv, len = seg->len;
      wait(sh.meta_full[par], (n_seg >> 1) & 1);  // nanpos is set
      for (int t = seg->tile0; t < tile1; ++t, ++k) {
        const int pos0 = t * kTile, pos = pos0 + t_in;
        const unsigned char* from = v_tiles + slot * L::kTileBytes;
        unsigned char* to = v_half + (k & 1) * L::kHalfBytes;
        wait(sh.v_full[slot], round & 1);
        uint4 c[D / 16];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) c[i] = *reinterpret_cast<const uint4*>(from + swizzled<D>(t_in, i * 16));
        warp_arrive(sh.v_empty[slot]);
        if (++slot == a.ring) slot = 0, ++round;
        if (pos0 + kTile > min(kv, len)) {
          if (pos >= len) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) c[i] = make_uint4(0, 0, 0, 0);
          } else if (pos >= kv) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
              for (int j = 0; j < 4; ++j)
                for (int e = 0; e < 4; ++e)
                  if (((w[j] >> (8 * e)) & 0x7F) == 0x7F) {
                    w[j] &= ~(0xFFu << (8 * e));
                    atomicMin(&sh.nanpos[par][i * 16 + j * 4 + e], pos);
                  }
              c[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        if (k >= 2) wait(sh.pv_done[k & 1], ((k >> 1) - 1) & 1);
        // rows of 64 values (128 bytes), swizzled; the two halves of D one after the other
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint4 q = c[i >> 1];
          const uint32_t lo = (i & 1) ? q.z : q.x, hi = (i & 1) ? q.w : q.y;
          const uint4 h = make_uint4(tc::f16x2_of_e4m3x2(lo & 0xFFFFu), tc::f16x2_of_e4m3x2(lo >> 16),
                                     tc::f16x2_of_e4m3x2(hi & 0xFFFFu), tc::f16x2_of_e4m3x2(hi >> 16));
          *reinterpret_cast<uint4*>(to + (i >> 3) * (kTile * 128) + t_in * 128 + (((i & 7) ^ (t_in & 7)) << 4)) = h;
        }
        tc::fence_smem();
        warp_arrive(sh.f_full[k & 1]);
      }
      warp_arrive(sh.l_full[par]);
      leave(n_seg);
    }
  } else if (warp < 16) {
    // ------------------------------------------------------------- Q and O
    tc::fewer_registers<kRegsOutput>();
    const int ot = tid - 384, ow = ot >> 5;
    const int d = D == 128 ? ot : 16 * ow + (lane & 15);
    const bool owns = D == 128 || lane < 16;
    constexpr int kVec = D / 16;  // 16-byte loads of half a row
    uint4 qv[kVec];
    const int qr = ot >> 1, half = ot & 1;  // two threads a row of Q
    auto load_q = [&](const Segment& s) {
      if (qr < s.rows) {
        const int row = s.row0 + qr;
        const uint4* p = reinterpret_cast<const uint4*>(a.q + (s.q0 + row / G) * a.q_stride + (s.h * G + row % G) * D +
                                                        half * (D / 2));
#pragma unroll
        for (int i = 0; i < kVec; ++i) qv[i] = __ldg(p + i);
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) qv[i] = make_uint4(0, 0, 0, 0);
      }
    };
    auto store_q = [&](const Segment& s, int par) {
      if (qr < (s.rows + 15) / 16 * 16) {
        float amax = 0.f;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          float f[8];
          unpack16<__nv_bfloat16>(qv[i], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            bad |= !isfinite(f[e]);
            amax = fmaxf(amax, fabsf(f[e]));
          }
        }
        const uint32_t pair = 3u << (lane & 30);
        amax = fmaxf(amax, __shfl_xor_sync(pair, amax, 1));
        bad = __shfl_xor_sync(pair, static_cast<int>(bad), 1) || bad;
        const float sc = pow2_scale(amax), inv = bad ? 0.f : pow2_inverse(sc);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          float f[8];
          uint32_t hw[2] = {0, 0}, lw[2] = {0, 0};
          if (!bad) {
            unpack16<__nv_bfloat16>(qv[i], f);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float u = f[e] * inv, v = f[e + 1] * inv;
              const float uh = top4(u), vh = top4(v);
              hw[e >> 2] |= tc::e4m3x2(uh, vh) << (8 * (e & 2));
              lw[e >> 2] |= tc::e4m3x2(u - uh, v - vh) << (8 * (e & 2));
            }
          }
          // 8 rows x 16 bytes lie together, then the rows' next 16 bytes
          const int at_x = half * (D / 2) + i * 8;
          const int at = (qr >> 3) * (8 * D) + (at_x >> 4) * 128 + (qr & 7) * 16 + (at_x & 15);
          *reinterpret_cast<uint2*>(q_hi + at) = make_uint2(hw[0], hw[1]);
          *reinterpret_cast<uint2*>(q_lo + at) = make_uint2(lw[0], lw[1]);
        }
        if (half == 0) {
          sh.qs[par][qr] = bad ? __uint_as_float(0x7FFFFFFFu) : (sc > 0.f ? sc : 1.f);
          sh.limit[par][qr] = qr < s.rows ? min(s.kv + (s.row0 + qr) / G, s.len - 1) : -1;
        }
      }
      sh.nanpos[par][ot] = 0x7FFFFFFF;
      tc::fence_smem();
      warp_arrive(sh.q_full);
      warp_arrive(sh.meta_full[par]);
    };
    const Segment* nxt = segment(0);
    if (nxt != nullptr) {
      load_q(*nxt);
      store_q(*nxt, 0);
    }
    for (int n_seg = 0;; ++n_seg) {
      if (named_any(3, 128, nxt == nullptr)) break;
      const int par = n_seg & 1;
      const Segment seg = *nxt;
      nxt = segment(n_seg + 1);
      if (nxt != nullptr) {
        load_q(*nxt);
        wait(sh.q_empty, n_seg & 1);
        store_q(*nxt, par ^ 1);
      }
      wait(sh.l_full[par], (n_seg >> 1) & 1);
      const bool by_rows = seg.rows > kHalfRows;
      const bool whole = seg.tile0 == 0 && seg.tile1 == seg.tiles;
      if (ot < seg.rows) {
        // a group whose sum is 0 has nothing, whatever its reference and O
        const int half_rows = by_rows ? (seg.rows + 15) / 16 * 8 : kAttnRows;
        const int r = ot % half_rows, own_grp = ot / half_rows;
        float s[2] = {0.f, 0.f}, m[2] = {0.f, 0.f}, M = -INFINITY;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (by_rows && g != own_grp) continue;
#pragma unroll
          for (int w = 0; w < 4; ++w) s[g] += sh.lsum[par][g * 4 + w][r];
          m[g] = sh.mrun[par][g][r];
          if (s[g] != 0.f) M = fmaxf(M, m[g]);
        }
        float f[2], sum = 0.f;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const float w = s[g] != 0.f ? tc::ex2(m[g] - M) : 0.f;
          sum += w * s[g];
          f[g] = s[g] != 0.f ? w * sh.vref[par][g] : 0.f;
        }
        if (by_rows) f[0] += f[1];  // one of them
        if (whole) sum = sum == 0.f ? 0.f : 1.f / sum;
        sh.fin[ot] = make_float4(f[0], f[1], sum, M);
      }
      named_barrier(3, 128);
      wait(sh.o_full[par], (n_seg >> 1) & 1);
      tc::fence_after();
      const int nan_at = sh.nanpos[par][d];
      const int slot = static_cast<int>(blockIdx.x) * 2 + (n_seg == 0 ? 0 : 1);
      float* rec = a.partial + static_cast<long long>(slot) * kPartialFloats;
      const uint32_t o_at = tmem + (static_cast<uint32_t>(ow * 32) << 16) + (2 + par) * kAttnRows;
      int tok = seg.row0 / G, g = seg.row0 % G;  // of row r
      __nv_bfloat16* dst = a.out + (static_cast<long long>(seg.q0 + tok) * a.Hq + seg.h * G + g) * D + d;
      const long long next_tok = static_cast<long long>(a.Hq - (G - 1)) * D;  // from a token's last head to the next's first
      for (int c = 0; c * 8 < seg.rows; ++c) {
        float o[8], o2[8];
        tc::ld8(o_at + c * 8, o);
        if (!by_rows) tc::ld8(o_at + kHalfRows + c * 8, o2);
        tc::wait_ld();
        tc::ready(o);
        if (!by_rows) tc::ready(o2);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int r = c * 8 + e;
          if (r < seg.rows) {
            const float4 f = sh.fin[r];
            float v = f.x != 0.f ? o[e] * f.x : 0.f;
            if (!by_rows && f.y != 0.f) v = fmaf(o2[e], f.y, v);
            if (nan_at <= seg.kv + tok) v = __uint_as_float(0x7FFFFFFFu);
            if (whole) {
              if (owns) *dst = __float2bfloat16_rn(v * f.z);
            } else if (owns) {
              rec[r * D + d] = v;
            }
            if (++g == G) {
              g = 0;
              ++tok;
              dst += next_tok;
            } else {
              dst += D;
            }
          }
        }
      }
      tc::fence_before();
      warp_arrive(sh.o_empty[par]);
      if (!whole) {
        if (ot < seg.rows) {
          rec[kAttnRows * 128 + ot] = sh.fin[ot].w;
          rec[kAttnRows * 128 + kAttnRows + ot] = sh.fin[ot].z;
        }
        // the last of the item's CTAs joins the parts
        const long long c0 = seg.first / chunk, c1 = (seg.first + seg.tiles - 1) / chunk;
        __threadfence();
        named_barrier(3, 128);
        if (ot == 0) sh.last = ptx::atom_add_acq_rel(a.counters + c0, 1u) == static_cast<uint32_t>(c1 - c0);
        named_barrier(3, 128);
        if (sh.last) {
          __threadfence();
          const int pieces = static_cast<int>(c1 - c0) + 1;
          const int first_slot = static_cast<int>(c0) * 2 + (seg.first % chunk == 0 ? 0 : 1);
          auto record = [&](int p) {
            return a.partial + static_cast<long long>(p == 0 ? first_slot : (c0 + p) * 2) * kPartialFloats;
          };
          constexpr int E = D / 32;  // a lane's values
          for (int r4 = 0; r4 < seg.rows; r4 += 16) {
            // rows r4 + ow, + 4, + 8, + 12 at once, for their loads' sake
            float M[4], sum[4], acc[4][E];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              M[j] = -INFINITY;
              sum[j] = 0.f;
#pragma unroll
              for (int i = 0; i < E; ++i) acc[j][i] = 0.f;
            }
            for (int p0 = 0; p0 < pieces; p0 += 32) {
              // a lane for each piece: its references and sums
              float m[4], n[4], w[4];
              const float* q = record(min(p0 + lane, pieces - 1)) + kAttnRows * 128 + r4 + ow;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const bool in = p0 + lane < pieces && r4 + ow + 4 * j < seg.rows;
                m[j] = in ? __ldcg(q + 4 * j) : 0.f;
                n[j] = in ? __ldcg(q + kAttnRows + 4 * j) : 0.f;
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float M_new = fmaxf(M[j], tc::warp_max(n[j] != 0.f ? m[j] : -INFINITY));
                const float f = M[j] > -INFINITY ? tc::ex2(M[j] - M_new) : 0.f;
                w[j] = n[j] != 0.f ? tc::ex2(m[j] - M_new) : 0.f;
                M[j] = M_new;
                float part = w[j] * n[j];
#pragma unroll
                for (int s = 16; s > 0; s >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, s);
                sum[j] = fmaf(sum[j], f, part);
#pragma unroll
                for (int i = 0; i < E; ++i) acc[j][i] *= f;
              }
              const int here = min(32, pieces - p0);
#pragma unroll 2
              for (int p = 0; p < here; ++p) {
                const float* y = record(p0 + p) + (r4 + ow) * D + lane * E;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float wp = __shfl_sync(0xFFFFFFFFu, w[j], p);
                  if (r4 + ow + 4 * j < seg.rows) {
                    float v[E];
                    if constexpr (D == 128) {
                      const float4 z = __ldcg(reinterpret_cast<const float4*>(y + 4 * j * D));
                      v[0] = z.x, v[1] = z.y, v[2] = z.z, v[3] = z.w;
                    } else {
                      const float2 z = __ldcg(reinterpret_cast<const float2*>(y + 4 * j * D));
                      v[0] = z.x, v[1] = z.y;
                    }
#pragma unroll
                    for (int i = 0; i < E; ++i) acc[j][i] = fmaf(wp, v[i], acc[j][i]);
                  }
                }
              }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int row = seg.row0 + r4 + ow + 4 * j;
              if (r4 + ow + 4 * j >= seg.rows) break;
              const float inv = sum[j] == 0.f ? 0.f : 1.f / sum[j];
              uint32_t* to = reinterpret_cast<uint32_t*>(
                  a.out + (static_cast<long long>(seg.q0 + row / G) * a.Hq + seg.h * G + row % G) * D + lane * E);
#pragma unroll
              for (int i = 0; i < E; i += 2) {
                const __nv_bfloat162 y = __floats2bfloat162_rn(acc[j][i] * inv, acc[j][i + 1] * inv);
                to[i / 2] = *reinterpret_cast<const uint32_t*>(&y);
              }
            }
          }
          if (ot == 0) ptx::st_relaxed_u32(a.counters + c0, 0u);
        }
      }
      leave(n_seg);
    }
  } else {
    tc::fewer_registers<kRegsRest>();
    if (warp == 16) {
    // ------------------------------------------------------------- copies
    // A lane holds a block: 32 block ids, then their scales, are loaded at a
    // time, a batch of whole tiles ahead of the one in use.
    struct Batch {
      int h, tiles, pages;  // tiles of the batch, blocks of its segment from its first on
      int id;
      float ks, vs;
    } now, nxt;
    const int pages_per_tile = kTile >> a.bs_log2;
    int n_seg = -1, tile = 0, tile_end = 0, seg_b = 0, seg_h = 0, seg_pages = 0;
    bool more = true;
    const int per_batch = 32 / pages_per_tile;
    auto load_ids = [&](Batch& x) {
      x.tiles = 0;
      if (tile >= tile_end) {
        if (n_seg >= 0 && more) leave(n_seg);
        const Segment* s = more ? segment(++n_seg) : nullptr;
        if (s == nullptr) {
          more = false;
          return;
        }
        tile = s->tile0;
        tile_end = s->tile1;
        seg_b = s->b;
        seg_h = s->h;
        seg_pages = (s->len + a.bs - 1) >> a.bs_log2;
      }
      x.tiles = min(per_batch, tile_end - tile);
      x.h = seg_h;
      const int page0 = tile * pages_per_tile;
      x.pages = max(0, seg_pages - page0);
      x.id = -1;
      if (lane < x.pages && lane < x.tiles * pages_per_tile)
        x.id = __ldg(a.table + static_cast<long long>(seg_b) * a.max_blocks + page0 + lane);
      tile += x.tiles;
    };
    auto load_scales = [&](Batch& x) {
      x.ks = x.vs = 0.f;
      if (x.tiles > 0 && x.id >= 0 && x.id < a.num_blocks) {
        x.ks = __ldg(a.k_scale + static_cast<long long>(x.id) * a.H + x.h);
        x.vs = __ldg(a.v_scale + static_cast<long long>(x.id) * a.H + x.h);
      }
    };
    if (lane == 0) {
      tc::prefetch_map(&k_map);
      tc::prefetch_map(&v_map);
    }
    load_ids(now);
    load_scales(now);
    int slot = 0, round = 0, k = 0;
    while (now.tiles > 0) {
      load_ids(nxt);
      for (int i = 0; i < now.tiles; ++i, ++k) {
        const int pages = max(0, min(pages_per_tile, now.pages - i * pages_per_tile));
        const int src = (i * pages_per_tile + lane) & 31;
        const int id = __shfl_sync(0xFFFFFFFFu, now.id, src);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          if (round > 0) wait(kv ? sh.v_empty[slot] : sh.k_empty[slot], (round - 1) & 1);
          const uint32_t bar = ptx::smem_addr(kv ? &sh.v_full[slot] : &sh.k_full[slot]);
          if (lane == 0) ptx::mbar_arrive_expect_tx(bar, pages * a.bs * D);
          __syncwarp();
          if (lane < pages)
            tc::load_4d(ptx::smem_addr((kv ? v_tiles : k_tiles) + slot * L::kTileBytes + lane * a.bs * D),
                        kv ? &v_map : &k_map, 0, 0, now.h, id, bar);
        }
        if (++slot == a.ring) slot = 0, ++round;
        if (i == 0) load_scales(nxt);  // its ids have had a tile's time
        const int sr = k % kScaleRing;
        if (k >= kScaleRing) wait(sh.sc_empty[sr], (k / kScaleRing - 1) & 1);
        const float ks = __shfl_sync(0xFFFFFFFFu, now.ks, src), vs = __shfl_sync(0xFFFFFFFFu, now.vs, src);
        const float vmax = tc::warp_max(lane < pages_per_tile ? vs : 0.f);
        if (lane < pages_per_tile) {
          sh.scales[sr].ks[lane] = ks * a.scale_log2e;
          sh.scales[sr].vs[lane] = vs;
        }
        if (lane == 0) sh.scales[sr].vmax = vmax;
        warp_arrive(sh.sc_full[sr]);
      }
      now = nxt;
    }
    // no copy is in flight when the CTA ends: every slot used has been filled
    Waiter drain;
    const int used = round > 0 ? a.ring : slot;
    for (int i = 0; i < used; ++i) {
      drain(sh.k_full[i], (i < slot ? round : round - 1) & 1);
      drain(sh.v_full[i], (i < slot ? round : round - 1) & 1);
    }
    wait.dead |= drain.dead;
    } else if (warp == 17) {
      // --------------------------------------------------- first products
      const uint64_t swz = D == 128 ? tc::kSwizzle128 : tc::kSwizzle64;
      const uint64_t kd0 = tc::smem_desc(ptx::smem_addr(k_tiles), 16, 8 * D, swz);
      const uint64_t qd0 = tc::smem_desc(ptx::smem_addr(q_hi), 128, 8 * D, tc::kSwizzleNone);
      const uint64_t qd1 = tc::smem_desc(ptx::smem_addr(q_lo), 128, 8 * D, tc::kSwizzleNone);
      int k = 0, slot = 0, round = 0;
      for (int n_seg = 0;; ++n_seg) {
        const Segment* seg = segment(n_seg);
        if (seg == nullptr) break;
        const uint32_t is = tc::instr(kTile, (seg->rows + 15) / 16 * 16, false, false);
        const int tiles = seg->tile1 - seg->tile0;
        wait(sh.q_full, n_seg & 1);
        for (int i = 0; i < tiles; ++i, ++k) {
          const uint64_t kd = kd0 + slot * (L::kTileBytes / 16);
          const uint32_t dst = tmem + (k & 1) * kAttnRows;
          wait(sh.k_full[slot], round & 1);
          if (k >= 2) wait(sh.s_empty[k & 1], ((k >> 1) - 1) & 1);
          tc::fence_after();
          if (tc::elect()) {
#pragma unroll
            for (int j = 0; j < D / 32; ++j) tc::mma_e4m3(dst, kd + j * 2, qd0 + j * 16, is, j > 0);
#pragma unroll
            for (int j = 0; j < D / 32; ++j) tc::mma_e4m3(dst, kd + j * 2, qd1 + j * 16, is, true);
            tc::commit(ptx::smem_addr(&sh.s_full[k & 1]));
            tc::commit(ptx::smem_addr(&sh.k_empty[slot]));
            if (i + 1 == tiles) tc::commit(ptx::smem_addr(&sh.q_empty));
          }
          __syncwarp();
          if (++slot == a.ring) slot = 0, ++round;
        }
        leave(n_seg);
      }
      // all products are done before the tensor memory goes back
      Waiter drain;
      if (tc::elect()) tc::commit(ptx::smem_addr(&sh.done[0]));
      __syncwarp();
      drain(sh.done[0], 0);
      wait.dead |= drain.dead;
    } else if (warp == 18) {
      // -------------------------------------------------- second products
      const uint64_t vd0 = tc::smem_desc(ptx::smem_addr(v_half), kTile * 128, 1024, tc::kSwizzle128);
      const uint64_t pd0 = tc::smem_desc(ptx::smem_addr(p_at), 128, 16 * kTile, tc::kSwizzleNone);
      int k = 0;
      for (int n_seg = 0;; ++n_seg) {
        const Segment* seg = segment(n_seg);
        if (seg == nullptr) break;
        const int par = n_seg & 1;
        const bool by_rows = seg->rows > kHalfRows;
        const uint32_t io = tc::instr(D, (seg->rows + 15) / 16 * 16, true, true);
        const int tiles = seg->tile1 - seg->tile0;
        if (n_seg >= 2) wait(sh.o_empty[par], ((n_seg >> 1) - 1) & 1);
        for (int i = 0; i < tiles; ++i, ++k) {
          const uint64_t vd = vd0 + (k & 1) * (L::kHalfBytes / 16);
          const uint64_t pd = pd0 + (k & 1) * (L::p_bytes(a.rows) / 16);
          const uint32_t dst = tmem + (2 + par) * kAttnRows + (by_rows ? 0 : (k & 1) * kHalfRows);
          const bool add = i >= (by_rows ? 1 : 2);
          wait(sh.f_full[k & 1], (k >> 1) & 1);
          wait(sh.p_full[k & 1], (k >> 1) & 1);
          tc::fence_after();
          if (tc::elect()) {
#pragma unroll
            for (int j = 0; j < kTile / 16; ++j) tc::mma_f16(dst, vd + j * 128, pd + j * 16, io, add || j > 0);
            tc::commit(ptx::smem_addr(&sh.pv_done[k & 1]));
            if (i + 1 == tiles) tc::commit(ptx::smem_addr(&sh.o_full[par]));
          }
          __syncwarp();
        }
        leave(n_seg);
      }
      Waiter drain;
      if (tc::elect()) tc::commit(ptx::smem_addr(&sh.done[1]));
      __syncwarp();
      drain(sh.done[1], 0);
      wait.dead |= drain.dead;
    } else {
      // -------------------------------------------------- list of segments
      Walker walk(a, u0, u1, sh.b0, sh.ub0);
      for (int n_seg = 0;; ++n_seg) {
        if (n_seg >= kSegRing) wait(sh.seg_empty[n_seg % kSegRing], (n_seg / kSegRing - 1) & 1);
        Segment s;
        const bool more = walk.next(s);
        if (!more) s.tile1 = -1;
        if (lane == 0) sh.seg[n_seg % kSegRing] = s;
        warp_arrive(sh.seg_full[n_seg % kSegRing]);
        if (!more) break;
      }
    }
  }
  __syncwarp();
  if (wait.dead) atomicOr(a.err, SPECDEC_DEV_ERR_TIMEOUT);
  __syncthreads();
  if (warp == 17) tc::dealloc(tmem, kTmemCols);
}

}  // namespace specdec
