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
// number of 4 bits plus a remainder of 4, held 16 times its size so that e4m3's
// least step, 2^-9, is 2^-13 of it (exact to 2^-21 of the row's largest).
// The two are rows of one B operand, so K is read from shared memory once, and
// the softmax adds their columns: shared memory's 128 bytes a cycle, of which a
// tile takes most, are the next limit after HBM.
//
// Second product: f16 x f16.  An e4m3 V is exact in f16, and one group of
// warps turns V's tiles over while the softmax is at work; P, times its block's
// value scale over the largest met so far, in f16 has 11 bits down to 2^-20 of
// its reference and 2^-31 of it is lost.  (P as two e4m3
// numbers needs no such step, but loses what is below 2^-22 of the largest,
// which a faint tail after one strong position is, and costs twice the
// arithmetic a probability.)
//
// The reference of a row is its largest score when it was last looked for: in
// the first tile, and whenever a later score lies more than 2^9 above it.  So
// O stays in tensor memory, and most tiles need no search for a maximum.
//
// Four groups of four warps do the softmax, a group 16 rows of a tile: up to 16
// rows each takes every fourth tile, up to 32 a pair every second one, above
// that the rows of every tile are divided among them.  Groups of different
// tiles have references, sums and an O of their own, which the output warps
// add up.  A tile thus has the time of several (its steps are short and wait
// for one another), and a thread's scores and sums are 32 registers.
//
// The tiles of all requests, heads and row groups form one list that is cut
// into equal parts, one for each CTA; what a cut separates is joined by the
// CTA that finishes last, in the order of the parts.
//
// Bound by the cache's bytes while a part lasts: a tile of D = 128 is 32 KB, of
// which an SM's share of a copy's rate brings one in 0.74 us, and takes 0.67 us
// at 16 rows and 0.74 at 32; from 33 to 48 rows it takes 1.09 us and 1.14 at 64,
// from HBM or L2 alike: there the softmax is next.
// From one (request, head) to the next some 7 us pass in which the next first
// tile's search, the last products and O's way out are only partly covered;
// that is what keeps many short parts from HBM's rate.  Measured: 64 requests
// of up to 5 tokens over up to 8000 positions (598 MB) 149 us, 4.0 TB/s; one of 2
// over 131000 (269 MB) 61 us, 4.4 TB/s; 256 of up to 8 over up to 4000 (1208 MB)
// 275 us, 4.4 TB/s; 32 of one over 18000 (665 MB) 116 us, 5.8 TB/s; one of one over
// 700 14 us.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "attention_cut.cuh"
#include "kv_kernels.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"
#include "waits.cuh"

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
  int32_t k_ring, v_ring;  // tiles of K and of V in shared memory
  int32_t rows;        // most rows of a tile: 16, 32 or 64
};

constexpr int kTile = 128;      // positions of a tile
constexpr int kAttnRows = 64;   // most rows of a tile
constexpr int kGroupRows = 16;  // of a softmax group
constexpr int kGroups = 4;
// Warps: 0-15 softmax (and what the CTA has to join), 16-23 V to f16 (four a
// half of D), 24-27 Q and O, 28 copies of K, 29 first products, 30 second
// products and the list of segments, 31 copies of V.
constexpr int kValueWarp = 16, kOutputWarp = 24, kCopyWarp = 28;
constexpr int kAttnThreads = 32 * 32;
// Registers a thread: 64 at launch, moved to where they are needed.  (40 for V
// spill in its loop: 66 us where one long request takes 60.)
constexpr int kRegsSoftmax = 72, kRegsValues = 48, kRegsOutput = 64, kRegsRest = 64;
static_assert(512 * kRegsSoftmax + 256 * kRegsValues + 128 * (kRegsOutput + kRegsRest) <= 64 * kAttnThreads,
              "the warpgroups' registers are those of the launch");
constexpr int kScaleRing = 8;
constexpr int kSegRing = 8;
constexpr int kSegAhead = 6;    // segments listed ahead of the second products'
constexpr int kMaxRing = 8;     // tiles of K, and of V, in shared memory
constexpr int kMaxPages = 8;    // blocks of a tile
constexpr uint32_t kTmemCols = 512;  // S (both halves of Q) in 256, O twice in 128
constexpr int kOutAt = 256;          // O's first column
constexpr int kPartialFloats = kAttnRows * 128 + 2 * kAttnRows;
// P = 2^kPScale at the reference score; a score may pass it by 2^kSlack
// before P would leave f16.
constexpr float kPScale = 64.f;
constexpr float kSlack = 9.f;

// Part of a (request, head, row group) that one CTA works on.  tile1 < 0 ends
// the list.
//
// How its tiles go over the softmax groups and their buffers goes by m, the
// 16s of rows: groups of different tiles are 4, 2 or 1 (by_log2), buffers of S
// and P 4 of up to 32 rows, or 2 (buf_log2).
struct Segment {
  int b, h, row0, rows;       // rows of this group
  int q0, kv, len;            // first token, positions before it, positions of the group
  int tile0, tile1, tiles;    // tiles of this part, and of the whole
  uint32_t first, end;        // units of the whole
  uint32_t per_tile;
  int m, by_log2, buf_log2;
  // columns of a buffer of S, and of one of a parity's Os
  __device__ int s_cols() const { return 256 >> buf_log2; }
  __device__ int o_cols() const { return kAttnRows >> by_log2; }
  // Arrivals of a group (or of each of its warps): all of a tile's make 4 (16).
  __device__ uint32_t weight(int part) const { return m == 3 ? (part == 0 ? 2 : 1) : (m == 1 ? 4 : m == 2 ? 2 : 1); }
};

// Parities of four barriers that are used in turn, buffer i % buffers for tile
// i of a segment; what every role of the CTA knows without asking.
struct Turns {
  uint32_t bits = 0;
  __device__ __forceinline__ uint32_t of(int i, int buf_log2) const {
    return ((bits >> (i & ((1 << buf_log2) - 1))) ^ static_cast<uint32_t>(i >> buf_log2)) & 1;
  }
  __device__ __forceinline__ void pass(int tiles, int buf_log2) {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int uses = (tiles + (1 << buf_log2) - 1 - b) >> buf_log2;  // (not past the last buffer)
      if (b < 1 << buf_log2) bits ^= static_cast<uint32_t>(uses & 1) << b;
    }
  }
};

// Goes through the segments of units [u, end).
struct Walker {
  const AttnArgs& a;
  uint32_t u, end, ub;  // ub: first unit of request b
  uint32_t per_head;
  int b, G, q0, q, kv;

  __device__ Walker(const AttnArgs& args, uint32_t u0, uint32_t u1, int b0, uint32_t ub0)
      : a(args), u(u0), end(u1), ub(ub0), per_head(0), b(b0 - 1), G(args.Hq / args.H), q0(0), q(0), kv(0) {}
  // positions of the row group that ends before row `row_end`
  static __device__ __forceinline__ int length(const AttnArgs& a, int kv, int G, int row_end) {
    const long long n = static_cast<long long>(kv) + (row_end - 1) / G + 1;
    return static_cast<int>(max(0LL, min(n, static_cast<long long>(a.max_blocks) << a.bs_log2)));
  }
  static __device__ __forceinline__ int tiles_of(int len) { return max(1, (len + kTile - 1) / kTile); }
  static __device__ __forceinline__ uint32_t units_per_head(const AttnArgs& a, int kv, int G, int q) {
    uint32_t n = 0;
#pragma unroll 1
    for (int r = 0; r < q * G; r += a.rows) {
      const int row_end = min(q * G, r + a.rows);
      n += tiles_of(length(a, kv, G, row_end)) * tile_cost(row_end - r) + kItemCost;
    }
    return n;
  }
  static __device__ __forceinline__ void request(const AttnArgs& a, int b, int& q0, int& q, int& kv) {
    q0 = max(0, min(__ldg(a.cu_tokens + b), a.T));
    const int q1 = max(0, min(__ldg(a.cu_tokens + b + 1), a.T));
    q = max(0, q1 - q0);
    kv = min(__ldg(a.kv_len + b), a.max_blocks << a.bs_log2);  // (positions behind the row's end: sums with it stay in 32 bits)
  }
  __device__ bool next(Segment& s) {
#pragma unroll 1
    while (u < end) {
#pragma unroll 1
      while (u - ub >= per_head * a.H) {
        ub += per_head * a.H;
        ++b;
        request(a, b, q0, q, kv);
        per_head = units_per_head(a, kv, G, q);
      }
      uint32_t rem = u - ub, cost, per_tile;
      s.b = b;
      s.h = static_cast<int>(rem / per_head);
      rem -= s.h * per_head;
      s.q0 = q0;
      s.kv = kv;
      s.row0 = 0;
#pragma unroll 1
      for (;; s.row0 += a.rows) {
        const int row_end = min(q * G, s.row0 + a.rows);
        s.rows = row_end - s.row0;
        s.len = length(a, kv, G, row_end);
        s.tiles = tiles_of(s.len);
        per_tile = tile_cost(s.rows);
        cost = s.tiles * per_tile + kItemCost;
        if (rem < cost) break;
        rem -= cost;
      }
      s.first = u - rem;
      s.end = s.first + cost;
      s.per_tile = per_tile;
      const uint32_t to = min(cost, rem + (end - u));
      s.tile0 = tiles_before(rem, per_tile, s.tiles);
      s.tile1 = tiles_before(to, per_tile, s.tiles);
      u += to - rem;
      if (s.tile0 >= s.tile1) continue;  // a cut before the first or after the last tile
      s.m = (s.rows + 15) / 16;
      s.by_log2 = s.m == 1 ? 2 : (s.m == 2 ? 1 : 0);
      s.buf_log2 = s.m <= 2 ? 2 : 1;
      return true;
    }
    return false;
  }
};

struct ScaleEntry {
  float ks[kMaxPages];   // key scale times the scores' factor
  float vs[kMaxPages];   // value scale
  float vmax;            // the tile's largest
};

// What the output warps know of a row.
struct alignas(16) RowOut {
  float4 f;     // factors of the groups' Os
  int32_t sees; // its last position
  int32_t at;   // its output, from the first row's token's first head of the group on
  float sum, ref;
};

// An item whose last part this CTA has finished.
struct Join {
  uint32_t cta0;  // of the first part
  int32_t pieces, row0, rows, q0, h;
};

struct AttnShared {
  uint64_t k_full[kMaxRing], k_empty[kMaxRing], v_full[kMaxRing], v_empty[kMaxRing];
  uint64_t s_full[4], s_empty[4], p_full[4], pv_done[4], f_full[2], f_empty[2], o_full[2], o_empty[2];
  uint64_t q_full, q_empty, meta_full[2], l_full[2], out_done;
  uint64_t sc_full[kScaleRing], sc_empty[kScaleRing], seg_full[kSegRing], seg_empty[kSegRing], done[2];
  uint32_t tmem;
  int32_t b0;
  uint32_t ub0;
  Segment seg[kSegRing];
  uint32_t part[32];
  alignas(16) float2 col[kGroups][kGroupRows];  // {row scale, reference} of each group's rows
  float wmax[kGroups][4][kGroupRows];  // a warp's largest score of each of its group's rows
  float fac[kGroups][kGroupRows];      // factors from a row's reference to its next
  float qs[2][kAttnRows];
  int32_t limit[2][kAttnRows];         // last position a row attends to
  alignas(16) float lsum[2][kGroups][kGroupRows][4];  // sums of the softmax warps
  float mrun[2][kGroups][kGroupRows];  // and their groups' references
  float vref[2][kGroups];
  RowOut out[kAttnRows];
  int32_t nanpos[2][128];              // first new position whose value is NaN in a dimension
  ScaleEntry scales[kScaleRing];
  Join join[2];  // of the item begun before this CTA's part, and of its last
  int32_t joins;
};

// One warp of a group polls a barrier, with pauses, and the others wait for it
// at a hardware barrier; where a group meets at one, one thread arrives for it.
// An SM's barrier operations take 5 to 8 cycles each, one after the other.
__device__ __forceinline__ void arrive(uint64_t& bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(ptx::smem_addr(&bar)), "r"(n) : "memory");
}
// Arrivals for the warp, after what all its threads did before.
__device__ __forceinline__ void warp_arrive(uint64_t& bar, uint32_t n = 1) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) arrive(bar, n);
}

// Q's remainder is held so many times its size (of 448 it is at most 16: 256).
constexpr float kRest = 16.f;

// Byte x of row t in a tile of K or V (rows of D bytes) as the copies swizzle it.
template <int D>
__device__ __forceinline__ int swizzled(int t, int x) {
  return D == 128 ? t * 128 + (x ^ ((t & 7) << 4)) : t * 64 + (x ^ (((t >> 1) & 3) << 4));
}

// Sums of 16 values over the warp: lane i gets that of value i >> 1.
__device__ __forceinline__ float warp_sums16(const float* v) {
  const int lane = threadIdx.x & 31;
  float a[8], b[4], c[2];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool up = lane & 16;
    a[i] = (up ? v[i + 8] : v[i]) + __shfl_xor_sync(0xFFFFFFFFu, up ? v[i] : v[i + 8], 16);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool up = lane & 8;
    b[i] = (up ? a[i + 4] : a[i]) + __shfl_xor_sync(0xFFFFFFFFu, up ? a[i] : a[i + 4], 8);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool up = lane & 4;
    c[i] = (up ? b[i + 2] : b[i]) + __shfl_xor_sync(0xFFFFFFFFu, up ? b[i] : b[i + 2], 4);
  }
  const bool up = lane & 2;
  const float s = (up ? c[1] : c[0]) + __shfl_xor_sync(0xFFFFFFFFu, up ? c[0] : c[1], 2);
  return s + __shfl_xor_sync(0xFFFFFFFFu, s, 1);
}

template <int D>
struct AttnLayout {
  static constexpr int kTileBytes = kTile * D;       // of K or V
  static constexpr int kHalfBytes = kTile * D * 2;   // of V in f16
  static __host__ __device__ int q_bytes(int rows) { return rows * D; }          // of one half
  // of all buffers: four of up to 32 rows or two of 64
  static __host__ __device__ int p_bytes(int rows) { return (rows <= 32 ? 4 * rows : 2 * rows) * kTile * 2; }
  static __host__ __device__ int tiles_at() { return (static_cast<int>(sizeof(AttnShared)) + 1023) / 1024 * 1024; }
  static __host__ __device__ int bytes(int tiles, int rows) {
    return tiles_at() + tiles * kTileBytes + 2 * kHalfBytes + 2 * q_bytes(rows) + p_bytes(rows);
  }
};

template <int D>
__global__ void __launch_bounds__(kAttnThreads, 1)
    attention_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
  using L = AttnLayout<D>;
  // (The kernel has no other shared memory, so this begins where an SM's does,
  // past the 1 KB that the system keeps.)
  extern __shared__ __align__(1024) unsigned char base[];
  AttnShared& sh = *reinterpret_cast<AttnShared*>(base);
  unsigned char* k_tiles = base + L::tiles_at();
  unsigned char* v_tiles = k_tiles + a.k_ring * L::kTileBytes;
  unsigned char* v_half = v_tiles + a.v_ring * L::kTileBytes;
  unsigned char* q_at = v_half + 2 * L::kHalfBytes;
  unsigned char* p_at = q_at + 2 * L::q_bytes(a.rows);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = a.Hq / a.H;

  if (tid == 0) {
    auto init = [](uint64_t& bar, uint32_t n) { ptx::mbar_init(ptx::smem_addr(&bar), n); };
    for (int i = 0; i < kMaxRing; ++i) {
      init(sh.k_full[i], 1);
      init(sh.k_empty[i], 1);
      init(sh.v_full[i], 1);
      init(sh.v_empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      init(sh.s_full[i], 1);
      init(sh.s_empty[i], 4);
      init(sh.p_full[i], 16);
      init(sh.pv_done[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      init(sh.f_full[i], 8);
      init(sh.f_empty[i], 1);
      init(sh.o_full[i], 1);
      init(sh.o_empty[i], 4);
      init(sh.meta_full[i], 4);
      init(sh.l_full[i], 24);
    }
    for (int i = 0; i < kScaleRing; ++i) {
      init(sh.sc_full[i], 2);
      init(sh.sc_empty[i], 4);
    }
    init(sh.q_full, 4);
    init(sh.out_done, 4);
    init(sh.q_empty, 1);
    init(sh.done[0], 1);
    init(sh.done[1], 1);
    for (int i = 0; i < kSegRing; ++i) {
      init(sh.seg_full[i], 1);
      init(sh.seg_empty[i], 32);
    }
    ptx::fence_mbarrier_init();
    sh.b0 = 0;
    sh.ub0 = 0;
    sh.joins = 0;
  }
  if (warp == kCopyWarp) tc::alloc(ptx::smem_addr(&sh.tmem), kTmemCols);

  // Units of all requests, and where this CTA's begin.
  uint32_t u0, u1, chunk;
  {
    const int per = (a.B + kAttnThreads - 1) / kAttnThreads;
    const int lo = min(a.B, tid * per), hi = min(a.B, lo + per);
    uint32_t before = 0, mine = 0;
    bool bad = false;
    // first the sum of this thread's requests, then the request of unit u0
    // where it is among them (sums stay at the largest int, which requests that
    // do not overlap cannot reach: the call is refused before)
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      uint32_t at = before;
#pragma unroll 1
      for (int b = lo; b < hi; ++b) {
        int q0, q, kv;
        Walker::request(a, b, q0, q, kv);
        const uint32_t n = Walker::units_per_head(a, kv, G, q) * a.H;
        if (pass == 1 && at <= u0 && u0 < at + n) {
          sh.b0 = b;
          sh.ub0 = at;
        }
        at = capped_sum(at, n);
        const int first = __ldg(a.cu_tokens + b), end = __ldg(a.cu_tokens + b + 1);
        bad |= first < 0 || end < first || end > a.T;
      }
      if (pass == 1) break;
      mine = at;
      uint32_t s = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, s, d);
        if (lane >= d) s = capped_sum(s, o);
      }
      if (lane == 31) sh.part[warp] = s;
      __syncthreads();
      // a lane for each warp
      const uint32_t w = lane < kAttnThreads / 32 ? sh.part[lane] : 0;
      // requests that overlap may have more units than can be counted: none then
      const unsigned long long all = (static_cast<unsigned long long>(__reduce_add_sync(0xFFFFFFFFu, w >> 16)) << 16) +
                                     __reduce_add_sync(0xFFFFFFFFu, w & 0xFFFFu);
      const uint32_t total = all < 0x7FFFFFFFull ? static_cast<uint32_t>(all) : 0;
      bad |= all >= 0x7FFFFFFFull;
      before = s - mine + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? w : 0);
      chunk = max((total + gridDim.x - 1) / gridDim.x, static_cast<uint32_t>(kLeastCost));
      u0 = min(static_cast<unsigned long long>(total), static_cast<unsigned long long>(blockIdx.x) * chunk);
      u1 = min(total, u0 + chunk);
      if (u0 >= u1 || before > u0 || u0 >= before + mine) break;
    }
    if (bad && blockIdx.x == 0) atomicOr(a.err, SPECDEC_DEV_ERR_SEGMENT);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
  }
  const uint32_t tmem = sh.tmem;
  Waiter wait;
  // The n-th segment, or null at the list's end; and the warp is done with it.
  auto segment = [&](int n) -> const Segment* {
    wait(sh.seg_full[n % kSegRing], (n / kSegRing) & 1);
    if (__any_sync(0xFFFFFFFFu, wait.dead())) wait.looks = 0;
    const Segment* s = &sh.seg[n % kSegRing];
    return wait.dead() || s->tile1 < 0 ? nullptr : s;
  };
  // bytes of a buffer of P
  auto p_stride = [&](int buf_log2) { return (buf_log2 == 2 ? min(a.rows, 32) : kAttnRows) * (kTile * 2); };
  auto leave = [&](int n) { warp_arrive(sh.seg_empty[n % kSegRing]); };

  if (warp < kValueWarp) {
    // ------------------------------------------------------------ softmax
    // A thread has one position and the 16 rows of its group.
    tc::more_registers<kRegsSoftmax>();
    const int grp = warp >> 2, t_in = tid & 127, page = t_in >> a.bs_log2;
    const bool leader = (warp & 3) == 0;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    float x[kGroupRows], l[kGroupRows];
    const float4* col = reinterpret_cast<const float4*>(sh.col[grp]);
    Turns turns;
    uint32_t k0 = 0;  // tiles of the segments before
    for (int n_seg = 0;; ++n_seg) {
      const Segment* seg = segment(n_seg);
      // (and the last segment's rows are no longer read)
      if (named_any(1 + grp, 128, seg == nullptr)) break;
      const int par = n_seg & 1;
      const int by_log2 = seg->by_log2, buf_log2 = seg->buf_log2, step = 1 << by_log2;
      const int part = grp & ((kGroups >> by_log2) - 1), turn = grp >> (2 - by_log2);
      const int r0 = part * kGroupRows;
      const uint32_t weight = seg->weight(part);
      const int tiles = seg->tile1 - seg->tile0, len = seg->len;
      const int all_see = seg->kv + seg->row0 / G;  // last position that all rows attend to
      const int pos_first = seg->tile0 * kTile;
      const uint32_t o_at = tmem + lanes + kOutAt + par * kAttnRows + turn * seg->o_cols() + r0;
      const uint32_t s_first = tmem + lanes + r0;
      const int s_cols = seg->s_cols(), p_bytes = p_stride(buf_log2), rest_at = 16 * seg->m;
      unsigned char* p_first = p_at + (r0 / 8) * (16 * kTile) + t_in * 16;
      float vref = 1.f, vinv = 1.f;
#pragma unroll
      for (int r = 0; r < kGroupRows; ++r) l[r] = 0.f;
      if (leader) wait(sh.meta_full[par], (n_seg >> 1) & 1);
      if (t_in < kGroupRows) sh.col[grp][t_in] = make_float2(sh.qs[par][r0 + t_in], 0.f);
      named_barrier(1 + grp, 128);
      bool first = true;
#pragma unroll 1
      for (int i = part < seg->m ? turn : tiles; i < tiles; i += step) {
        const uint32_t k = k0 + i;
        const int buf = i & ((1 << buf_log2) - 1), pos0 = pos_first + i * kTile, pos = pos0 + t_in;
        const uint32_t phase = turns.of(i, buf_log2);
        const bool masked = pos0 + kTile - 1 > all_see || pos0 + kTile > len;
        const ScaleEntry& sc = sh.scales[k % kScaleRing];
        if (leader) {
          wait(sh.sc_full[k % kScaleRing], (k / kScaleRing) & 1);
          wait(sh.s_full[buf], phase);
        }
        named_barrier(1 + grp, 128);
        tc::fence_after();
        const float ks = sc.ks[page], vs = sc.vs[page], vmax = sc.vmax;
        const uint32_t s_at = s_first + buf * s_cols;
        bool renew = first;
#pragma unroll 1
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
            for (int c = 0; c < kGroupRows; c += 8) {
              float v[8], rest[8], mine = -INFINITY;
              tc::ld8(s_at + c, v);
              tc::ld8(s_at + rest_at + c, rest);
              tc::wait_ld();
              tc::ready(v);
              tc::ready(rest);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                float y = fmaf(rest[e], 1.f / kRest, v[e]) * ks;
                if (masked && pos > sh.limit[par][r0 + c + e]) y = -INFINITY;
                y = tc::warp_max(y);
                if (lane == e) mine = y;
              }
              if (lane < 8) sh.wmax[grp][warp & 3][c + lane] = mine;
            }
            if (leader) {
              if (!first) wait(sh.pv_done[(i - step) & ((1 << buf_log2) - 1)], turns.of(i - step, buf_log2));  // O rests
            }
            tc::fence_after();
            named_barrier(1 + grp, 128);
            if (t_in < kGroupRows) {
              const float m = fmaxf(fmaxf(sh.wmax[grp][0][t_in], sh.wmax[grp][1][t_in]),
                                    fmaxf(sh.wmax[grp][2][t_in], sh.wmax[grp][3][t_in])) * sh.col[grp][t_in].x;
              const float was = sh.col[grp][t_in].y;
              const float now = first ? (m > -INFINITY ? m : 0.f) : fmaxf(was, m);
              sh.col[grp][t_in].y = now;
              sh.fac[grp][t_in] = tc::ex2(was - now);
            }
            named_barrier(1 + grp, 128);
            if (!first) {
#pragma unroll
              for (int r = 0; r < kGroupRows; ++r) l[r] *= sh.fac[grp][r];
              const float v_ratio = vref_was * vinv;
#pragma unroll 1
              for (int c = 0; c < kGroupRows; c += 8) {
                float o[8];
                tc::ld8(o_at + c, o);
                tc::wait_ld();
                tc::ready(o);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] *= sh.fac[grp][c + e] * v_ratio;
                tc::st8(o_at + c, o);
              }
              tc::wait_st();
              tc::fence_before();
            }
          }
          // scores over the rows' references
          float rest[kGroupRows];
          tc::ld8(s_at, x);
          tc::ld8(s_at + rest_at, rest);
          tc::ld8(s_at + 8, x + 8);
          tc::ld8(s_at + rest_at + 8, rest + 8);
          tc::wait_ld();
          tc::ready(x);
          tc::ready(x + 8);
          tc::ready(rest);
          tc::ready(rest + 8);
#pragma unroll
          for (int r = 0; r < kGroupRows; r += 2) {
            const float4 w = col[r >> 1];
            x[r] = fmaf(fmaf(rest[r], 1.f / kRest, x[r]) * ks, w.x, -w.y);
            x[r + 1] = fmaf(fmaf(rest[r + 1], 1.f / kRest, x[r + 1]) * ks, w.z, -w.w);
          }
          if (masked) {
#pragma unroll
            for (int r = 0; r < kGroupRows; ++r)
              if (pos > sh.limit[par][r0 + r]) x[r] = -INFINITY;
          }
          float top[2] = {x[0], x[1]};
#pragma unroll
          for (int r = 2; r < kGroupRows; ++r) top[r & 1] = fmaxf(top[r & 1], x[r]);
          // does P stay within f16 (and the sum within 32 bits)?
          const bool over = fmaxf(top[0], top[1]) > fminf(kSlack - __log2f(vs * vinv), 60.f) || vmax > 4.f * vref;
          // (and P's buffer has been read)
          if (leader) wait(sh.pv_done[buf], phase ^ 1);
          tc::fence_before();
          if (!named_any(1 + grp, 128, over && !renew)) break;
          renew = true;
        }
        if (leader && lane == 0) {  // all have read the scores and the scales
          arrive(sh.s_empty[buf], weight);
          arrive(sh.sc_empty[k % kScaleRing], weight);
        }
        first = false;
        const float vr = vs * vinv * kPScale;
        // probabilities
        uint32_t w[kGroupRows / 2];
#pragma unroll
        for (int r = 0; r < kGroupRows; r += 2) {
          const float p0 = tc::ex2(x[r]), p1 = tc::ex2(x[r + 1]);
          l[r] += p0;
          l[r + 1] += p1;
          w[r >> 1] = tc::f16x2(p0 * vr, p1 * vr);
        }
        unsigned char* p = p_first + buf * p_bytes;
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(p + 16 * kTile) = make_uint4(w[4], w[5], w[6], w[7]);
        tc::fence_smem();
        warp_arrive(sh.p_full[buf], weight);
      }
      k0 += tiles;
      turns.pass(tiles, buf_log2);
      // sums and references for the output warps
      const float s = warp_sums16(l);
      if ((lane & 1) == 0) sh.lsum[par][grp][lane >> 1][warp & 3] = s;
      if (t_in < kGroupRows) sh.mrun[par][grp][t_in] = sh.col[grp][t_in].y;
      if (t_in == 0) sh.vref[par][grp] = vref / kPScale;
      warp_arrive(sh.l_full[par]);
      leave(n_seg);
    }
    // The items that this CTA has finished: their parts are added up in their
    // order, a warp for 64 dimensions of a row.
    if (leader) wait(sh.out_done, 0);
    named_barrier(1 + grp, 128);
    const int joins = sh.joins;
#pragma unroll 1
    for (int i = 0; i < joins; ++i) {
      const Join& J = sh.join[i];
      auto record = [&](int p) {
        return a.partial + static_cast<size_t>((J.cta0 + p) * 2 + (p == 0 ? 1 : 0)) * kPartialFloats;
      };
#pragma unroll 1
      for (int task = warp; task < J.rows * (D / 64); task += kValueWarp) {
        const int r = task / (D / 64), x = task % (D / 64) * 64 + lane * 2;
        float M = -INFINITY, sum = 0.f, acc[2] = {0.f, 0.f};
#pragma unroll 1
        for (int p0 = 0; p0 < J.pieces; p0 += 32) {
          // a lane for each piece: its reference and sum
          const float* q = record(min(p0 + lane, J.pieces - 1)) + kAttnRows * 128 + r;
          const float m = __ldcg(q), n = p0 + lane < J.pieces ? __ldcg(q + kAttnRows) : 0.f;
          const float M_new = fmaxf(M, tc::warp_max(n != 0.f ? m : -INFINITY));
          const float f = M > -INFINITY ? tc::ex2(M - M_new) : 0.f, w = n != 0.f ? tc::ex2(m - M_new) : 0.f;
          M = M_new;
          float part = n != 0.f ? w * n : 0.f;
#pragma unroll
          for (int s = 16; s > 0; s >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, s);
          sum = fmaf(sum, f, part);
          acc[0] *= f;
          acc[1] *= f;
          const int here = min(32, J.pieces - p0);
#pragma unroll 8
          for (int p = 0; p < here; ++p) {
            const float wp = __shfl_sync(0xFFFFFFFFu, w, p);
            const float2 y = __ldcg(reinterpret_cast<const float2*>(record(p0 + p) + r * D + x));
            acc[0] = fmaf(wp, y.x, acc[0]);
            acc[1] = fmaf(wp, y.y, acc[1]);
          }
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int row = J.row0 + r, tok = row / G;
        *reinterpret_cast<__nv_bfloat162*>(a.out + (static_cast<long long>(J.q0 + tok) * a.Hq + J.h * G + row - tok * G) * D + x) =
            __floats2bfloat162_rn(acc[0] * inv, acc[1] * inv);
      }
    }
  } else if (warp < kOutputWarp) {
    // ------------------------------------------------------------ V to f16
    // A thread has one position, and half of its values.  Values past the last
    // position are no numbers of the request's: zeros.  New positions are not
    // seen by all rows: their NaN leave the product, where 0 times NaN would
    // spoil rows that do not see them, and are noted for the output.
    tc::fewer_registers<kRegsValues>();
    const int t_in = tid & 127, half = (warp - kValueWarp) >> 2;
    const bool leader = warp == kValueWarp;
    constexpr int kVec = D / 32;  // 16-byte loads of half a row
    // rows as the copies swizzle them, and rows of 64 f16 (128 bytes) as the
    // second product reads them, the two halves of D = 128 one after the other:
    // 16 bytes are where the row's number changes their own
    const uint32_t from_row = ptx::smem_addr(v_tiles) + (D == 128 ? t_in * 128 + (((t_in & 7) ^ (half * kVec)) << 4)
                                                                  : t_in * 64 + ((((t_in >> 1) & 3) ^ (half * kVec)) << 4));
    const uint32_t to_row = ptx::smem_addr(v_half) + t_in * 128 +
                            (D == 128 ? ((t_in & 7) << 4) + half * (kTile * 128) : ((t_in & 7) ^ (half * 4)) << 4);
    uint32_t k = 0;
    int slot = 0, round = 0;
    for (int n_seg = 0;; ++n_seg) {
      const Segment* seg = segment(n_seg);
      if (named_any(6, 256, seg == nullptr)) break;
      const int par = n_seg & 1, kv = seg->kv, len = seg->len, pos_end = seg->tile1 * kTile;
      if (leader) wait(sh.meta_full[par], (n_seg >> 1) & 1);  // nanpos is set
#pragma unroll 1
      for (int pos = seg->tile0 * kTile + t_in; pos < pos_end; pos += kTile, ++k) {
        const uint32_t from = from_row + slot * L::kTileBytes, to = to_row + (k & 1) * L::kHalfBytes;
        if (leader) wait(sh.v_full[slot], round & 1);
        named_barrier(6, 256);
        uint4 c[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) c[i] = tc::ld_shared(from ^ (i << 4));
        uint32_t nan = 0;
        if (pos - t_in + kTile > min(kv, len)) {
          const uint32_t keep = pos < len ? 0xFFFFFFFFu : 0;
#pragma unroll
          for (int i = 0; i < kVec; ++i) {
            c[i].x &= keep, c[i].y &= keep, c[i].z &= keep, c[i].w &= keep;
            nan |= tc::e4m3_nan(c[i].x) | tc::e4m3_nan(c[i].y) | tc::e4m3_nan(c[i].z) | tc::e4m3_nan(c[i].w);
          }
          nan = pos >= kv ? nan & 0x80808080u : 0;
        }
        if (leader && k >= 2) wait(sh.f_empty[k & 1], ((k >> 1) - 1) & 1);
        named_barrier(6, 256);
        if (leader && lane == 0) ptx::mbar_arrive(ptx::smem_addr(&sh.v_empty[slot]));
        if (++slot == a.v_ring) slot = 0, ++round;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t lo = j ? c[i].z : c[i].x, hi = j ? c[i].w : c[i].y;
            tc::st_shared(to ^ ((2 * i + j) << 4),
                          make_uint4(tc::f16x2_of_e4m3x2(lo), tc::f16x2_of_e4m3x2(lo >> 16), tc::f16x2_of_e4m3x2(hi),
                                     tc::f16x2_of_e4m3x2(hi >> 16)));
          }
        }
        if (nan) {
#pragma unroll 1
          for (int x = 0; x < D / 2; ++x) {
            const uint32_t at = (to ^ ((x >> 3) << 4)) + (x & 7) * 2;
            if ((tc::ld_shared_u16(at) & 0x7FFF) > 0x7C00) {
              tc::st_shared_u16(at, 0);
              atomicMin(&sh.nanpos[par][half * (D / 2) + x], pos);
            }
          }
        }
        tc::fence_smem();
        warp_arrive(sh.f_full[k & 1]);
      }
      warp_arrive(sh.l_full[par]);
      leave(n_seg);
    }
  } else if (warp < kCopyWarp) {
    // ------------------------------------------------------------- Q and O
    tc::fewer_registers<kRegsOutput>();
    const int ot = tid - 32 * kOutputWarp, ow = ot >> 5;
    const int d = D == 128 ? ot : 16 * ow + (lane & 15);
    const bool owns = D == 128 || lane < 16;
    constexpr int kVec = D / 16;  // 16-byte loads of half a row
    uint4 qv[kVec];   // a thread's values of Q, then their codes and remainders
    float q_scale;    // of its row
    const int qr = ot >> 1, half = ot & 1;  // two threads a row of Q
    auto load_q = [&](const Segment& s) {
      const int row = s.row0 + min(qr, s.rows - 1);
      const uint4* p = reinterpret_cast<const uint4*>(a.q + (s.q0 + row / G) * a.q_stride + (s.h * G + row % G) * D +
                                                      half * (D / 2));
#pragma unroll
      for (int i = 0; i < kVec; ++i) qv[i] = __ldg(p + i);
    };
    auto convert_q = [&](const Segment& s) {
      // the largest magnitude's bits (bf16 in both halves; no number is above infinity)
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        top = __vmaxu2(top, __vmaxu2(qv[i].x & 0x7FFF7FFFu, qv[i].y & 0x7FFF7FFFu));
        top = __vmaxu2(top, __vmaxu2(qv[i].z & 0x7FFF7FFFu, qv[i].w & 0x7FFF7FFFu));
      }
      top = max(top >> 16, top & 0xFFFFu);
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      const bool bad = top >= 0x7F80u;
      const float sc = pow2_scale(__uint_as_float(top << 16)), inv = qr < s.rows && !bad ? pow2_inverse(sc) : 0.f;
      q_scale = bad ? __uint_as_float(0x7FFFFFFFu) : (sc > 0.f ? sc : 1.f);
      const uint32_t keep = bad ? 0 : 0xFFFFFFFFu;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        float f[8];
        unpack16<__nv_bfloat16>(make_uint4(qv[i].x & keep, qv[i].y & keep, qv[i].z & keep, qv[i].w & keep), f);
        // the nearest codes, and those of what they leave
        uint32_t hw[2] = {0, 0}, lw[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float u0 = f[2 * e] * inv, u1 = f[2 * e + 1] * inv;
          const uint32_t h = e4m3_pair(u0, u1);
          const float2 hf = e4m3_values(h);
          const uint32_t l = e4m3_pair((u0 - hf.x) * kRest, (u1 - hf.y) * kRest);
          hw[e >> 1] |= h << 16 * (e & 1);
          lw[e >> 1] |= l << 16 * (e & 1);
        }
        qv[i] = make_uint4(hw[0], hw[1], lw[0], lw[1]);
      }
    };
    auto store_q = [&](const Segment& s, int par) {
      if (qr < 16 * s.m) {
        // 8 rows x 16 bytes lie together, then the rows' next 16 bytes
        unsigned char* to = q_at + (qr >> 3) * (8 * D) + half * (D / 32 * 128) + (qr & 7) * 16;
#pragma unroll
        for (int i = 0; i < kVec; i += 2) {
          *reinterpret_cast<uint4*>(to + i / 2 * 128) = make_uint4(qv[i].x, qv[i].y, qv[i + 1].x, qv[i + 1].y);
          *reinterpret_cast<uint4*>(to + s.m * 16 * D + i / 2 * 128) = make_uint4(qv[i].z, qv[i].w, qv[i + 1].z, qv[i + 1].w);
        }
        if (half == 0) {
          sh.qs[par][qr] = q_scale;
          sh.limit[par][qr] = qr < s.rows ? min(s.kv + (s.row0 + qr) / G, s.len - 1) : -1;
        }
      }
      sh.nanpos[par][ot] = 0x7FFFFFFF;
      tc::fence_smem();
      warp_arrive(sh.q_full);
      warp_arrive(sh.meta_full[par]);
    };
    // Q is asked for two segments ahead and made one ahead, before this one's O.
    const Segment* next = segment(0);
    bool more = !named_any(5, 128, next == nullptr);
    if (more) load_q(*next);
    const Segment* at_seg = nullptr;
    for (int n_seg = -1;; ++n_seg) {
      const int par = n_seg & 1;
      const Segment* after = nullptr;
      bool more_after = false;
      if (more) {
        convert_q(*next);
        if (n_seg >= 0) wait(sh.q_empty, n_seg & 1, 200);
        store_q(*next, par ^ 1);
        after = segment(n_seg + 2);
        more_after = !named_any(5, 128, after == nullptr);
        if (more_after) load_q(*after);
      }
      if (n_seg < 0) {
        if (!more) break;
        at_seg = next;
        next = after;
        more = more_after;
        continue;
      }
      const Segment& seg = *at_seg;
      wait(sh.l_full[par], (n_seg >> 1) & 1, 200);
      const int by_tile = 1 << seg.by_log2, o_cols = seg.o_cols();
      const bool whole = seg.tile0 == 0 && seg.tile1 == seg.tiles;
      if (ot < seg.rows) {
        // a group whose sum is 0 has nothing, whatever its reference and O
        const int r = ot % kGroupRows, part = ot / kGroupRows, parts = kGroups >> seg.by_log2;
        float s[kGroups], m[kGroups], M = -INFINITY, f[kGroups], sum = 0.f;
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
          const int g = (j * parts + part) & (kGroups - 1);  // of turn j
          const float4 w = *reinterpret_cast<const float4*>(sh.lsum[par][g][r]);
          s[j] = j < by_tile ? (w.x + w.y) + (w.z + w.w) : 0.f;
          m[j] = s[j] != 0.f ? sh.mrun[par][g][r] : -INFINITY;
          f[j] = sh.vref[par][g];
          M = fmaxf(M, m[j]);
        }
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
          const float w = s[j] != 0.f ? tc::ex2(m[j] - M) : 0.f;
          sum = s[j] != 0.f ? fmaf(w, s[j], sum) : sum;
          f[j] = s[j] != 0.f ? w * f[j] : 0.f;
        }
        const float scale = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
        const int row = seg.row0 + ot, tok = row / G;
        RowOut& ro = sh.out[ot];
        ro.f = make_float4(f[0] * scale, f[1] * scale, f[2] * scale, f[3] * scale);
        ro.sees = seg.kv + tok;
        ro.at = ((tok - seg.row0 / G) * a.Hq + row - tok * G) * D;
        ro.sum = sum;
        ro.ref = M;
      }
      named_barrier(5, 128);
      wait(sh.o_full[par], (n_seg >> 1) & 1, 200);
      tc::fence_after();
      const int nan_at = sh.nanpos[par][d];
      // a CTA's records: of an item from before, and of one that begins here
      const int slot = static_cast<int>(blockIdx.x) * 2 + (seg.tile0 == 0 ? 1 : 0);
      float* rec = a.partial + static_cast<size_t>(slot) * kPartialFloats;
      __nv_bfloat16* dst = a.out + (static_cast<long long>(seg.q0 + seg.row0 / G) * a.Hq + seg.h * G) * D;
      const uint32_t o_at = tmem + (static_cast<uint32_t>(ow * 32) << 16) + kOutAt + par * kAttnRows;
      __nv_bfloat16* dst_d = dst + d;
      float* rec_d = rec + d;
#pragma unroll 1
      for (int c = 0; c < seg.rows; c += 8) {
        float v[8], f[8];
        int at[8];
        tc::ld8(o_at + c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = sh.out[c + e].f.x;
        tc::wait_ld();
        tc::ready(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = f[e] != 0.f ? v[e] * f[e] : 0.f;
#pragma unroll 1
        for (int j = 1; j < by_tile; ++j) {  // the other groups' Os
          float y[8];
          tc::ld8(o_at + j * o_cols + c, y);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = reinterpret_cast<const float*>(&sh.out[c + e].f)[j];
          tc::wait_ld();
          tc::ready(y);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = f[e] != 0.f ? fmaf(y[e], f[e], v[e]) : v[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int2 ro = *reinterpret_cast<const int2*>(&sh.out[c + e].sees);
          at[e] = ro.y;
          v[e] = nan_at <= ro.x ? __uint_as_float(0x7FFFFFFFu) : v[e];
        }
        const int rows = owns ? seg.rows - c : 0;
        if (whole) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e < rows) dst_d[at[e]] = __float2bfloat16_rn(v[e]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e < rows) rec_d[(c + e) * D] = v[e];
        }
      }
      tc::fence_before();
      warp_arrive(sh.o_empty[par]);
      if (!whole && ot < seg.rows) {
        rec[kAttnRows * 128 + ot] = sh.out[ot].ref;
        rec[kAttnRows * 128 + kAttnRows + ot] = sh.out[ot].sum;
      }
      // All have read sh.out and nanpos, which the next turn writes, and written
      // their part of the record.
      named_barrier(5, 128);
      if (!whole && ot == 0) {
        // the last of the item's CTAs joins the parts
        const ItemCtas on = item_ctas(seg.first, seg.end, seg.per_tile, seg.tiles, chunk);
        __threadfence();
        if (ptx::atom_add_acq_rel(a.counters + on.home, 1u) == on.c1 - on.c0) {
          ptx::st_relaxed_u32(a.counters + on.home, 0u);
          sh.join[sh.joins++] = Join{on.c0, static_cast<int>(on.c1 - on.c0) + 1, seg.row0, seg.rows, seg.q0, seg.h};
        }
      }
      leave(n_seg);
      if (!more) break;
      at_seg = next;
      next = after;
      more = more_after;
    }
    warp_arrive(sh.out_done);
  } else {
    tc::fewer_registers<kRegsRest>();
    if (warp == kCopyWarp || warp == kCopyWarp + 3) {
      // ------------------------------------------------------------- copies
      // A lane holds a block: 32 block ids, then their scales, are loaded at a
      // time, a batch of whole tiles ahead of the one in use.
      struct Batch {
        int h, tiles, pages;  // tiles of the batch, blocks of its segment from its first on
        int id;
        float scale;
      } now, nxt;
      const bool is_v = warp != kCopyWarp;
      const float* scales = is_v ? a.v_scale : a.k_scale;
      const CUtensorMap* map = is_v ? &v_map : &k_map;
      unsigned char* tiles = is_v ? v_tiles : k_tiles;
      uint64_t* full = is_v ? sh.v_full : sh.k_full;
      uint64_t* empty = is_v ? sh.v_empty : sh.k_empty;
      const int ring = is_v ? a.v_ring : a.k_ring;
      const int pages_log2 = 7 - a.bs_log2, pages_per_tile = 1 << pages_log2;
      int n_seg = -1, tile = 0, tile_end = 0, seg_b = 0, seg_h = 0, seg_pages = 0;
      bool more = true;
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
        x.tiles = min(32 >> pages_log2, tile_end - tile);
        x.h = seg_h;
        const int page0 = tile << pages_log2;
        x.pages = max(0, seg_pages - page0);
        x.id = -1;
        if (lane < x.pages && lane < x.tiles << pages_log2)
          x.id = __ldg(a.table + static_cast<long long>(seg_b) * a.max_blocks + page0 + lane);
        tile += x.tiles;
      };
      auto load_scales = [&](Batch& x) {
        x.scale = 0.f;
        if (x.tiles > 0 && x.id >= 0 && x.id < a.num_blocks) x.scale = __ldg(scales + static_cast<long long>(x.id) * a.H + x.h);
      };
      if (lane == 0) tc::prefetch_map(map);
      now.tiles = 0;
      int slot = 0, round = 0;
      uint32_t k = 0;
#pragma unroll 1
      for (;;) {
        load_ids(nxt);
        if (now.tiles == 0) load_scales(nxt);
#pragma unroll 1
        for (int i = 0; i < now.tiles; ++i, ++k) {
          const int first = i << pages_log2;
          const int pages = max(0, min(pages_per_tile, now.pages - first));
          if (round > 0) wait(empty[slot], (round - 1) & 1);
          const uint32_t bar = ptx::smem_addr(&full[slot]);
          const uint32_t dst = ptx::smem_addr(tiles + slot * L::kTileBytes);
          if (tc::elect()) ptx::mbar_arrive_expect_tx(bar, pages * a.bs * D);
          __syncwarp();
          int ids[kMaxPages];
#pragma unroll
          for (int j = 0; j < kMaxPages; ++j) ids[j] = __shfl_sync(0xFFFFFFFFu, now.id, (first + j) & 31);
          if (tc::elect()) {
#pragma unroll
            for (int j = 0; j < kMaxPages; ++j)
              if (j < pages) tc::load_4d(dst + j * a.bs * D, map, 0, 0, now.h, ids[j], bar);
          }
          __syncwarp();
          if (++slot == ring) slot = 0, ++round;
          if (i == 0) load_scales(nxt);  // its ids have had a tile's time
          const uint32_t sr = k % kScaleRing;
          if (k >= kScaleRing) wait(sh.sc_empty[sr], (k / kScaleRing - 1) & 1);
          const float scale = __shfl_sync(0xFFFFFFFFu, now.scale, (first + lane) & 31);
          if (is_v) {
            const float vmax = tc::warp_max(lane < pages_per_tile ? scale : 0.f);
            if (lane == 0) sh.scales[sr].vmax = vmax;
          }
          if (lane < pages_per_tile) (is_v ? sh.scales[sr].vs : sh.scales[sr].ks)[lane] = is_v ? scale : scale * a.scale_log2e;
          warp_arrive(sh.sc_full[sr]);
        }
        if (nxt.tiles == 0) break;
        now = nxt;
      }
      // no copy is in flight when the CTA ends: every slot used has been filled
      Waiter drain;
      const int used = round > 0 ? ring : slot;
      for (int i = 0; i < used; ++i) drain(full[i], (i < slot ? round : round - 1) & 1);
      if (drain.dead()) wait.looks = 0;
    } else if (warp == kCopyWarp + 1) {
      // --------------------------------------------------- first products
      const uint64_t swz = D == 128 ? tc::kSwizzle128 : tc::kSwizzle64;
      const uint64_t kd0 = tc::smem_desc(ptx::smem_addr(k_tiles), 16, 8 * D, swz);
      const uint64_t qd0 = tc::smem_desc(ptx::smem_addr(q_at), 128, 8 * D, tc::kSwizzleNone);
      int slot = 0, round = 0, was = 0;
      Turns turns;
      for (int n_seg = 0;; ++n_seg) {
        const Segment* seg = segment(n_seg);
        if (seg == nullptr) break;
        const uint32_t is = tc::instr(kTile, 32 * seg->m, false, false);
        const int tiles = seg->tile1 - seg->tile0, buf_log2 = seg->buf_log2, s_cols = seg->s_cols();
        wait(sh.q_full, n_seg & 1);
        if (seg->m != was) {
          // Other groups use the buffers now, or they lie elsewhere: the last
          // segment's second products are over first.  (So a group has seen
          // each use of a buffer since, as a wait for a parity needs.  O of the
          // segment before that has been drained: this Q is there.)
          if (n_seg > 0) wait(sh.o_full[(n_seg - 1) & 1], ((n_seg - 1) >> 1) & 1);
          was = seg->m;
        }
#pragma unroll 1
        for (int i = 0; i < tiles; ++i) {
          const uint64_t kd = kd0 + slot * (L::kTileBytes / 16);
          const int buf = i & ((1 << buf_log2) - 1);
          const uint32_t dst = tmem + buf * s_cols;
          wait(sh.k_full[slot], round & 1);
          wait(sh.s_empty[buf], turns.of(i, buf_log2) ^ 1);
          tc::fence_after();
          if (tc::elect()) {
#pragma unroll
            for (int j = 0; j < D / 32; ++j) tc::mma_e4m3(dst, kd + j * 2, qd0 + j * 16, is, j > 0);
            tc::commit(ptx::smem_addr(&sh.s_full[buf]));
            tc::commit(ptx::smem_addr(&sh.k_empty[slot]));
            if (i + 1 == tiles) tc::commit(ptx::smem_addr(&sh.q_empty));
          }
          __syncwarp();
          if (++slot == a.k_ring) slot = 0, ++round;
        }
        turns.pass(tiles, buf_log2);
        leave(n_seg);
      }
      // all products are done before the tensor memory goes back
      Waiter drain;
      if (tc::elect()) tc::commit(ptx::smem_addr(&sh.done[0]));
      __syncwarp();
      drain(sh.done[0], 0);
      if (drain.dead()) wait.looks = 0;
    } else {
      // -------------------------------------------------- second products
      const uint64_t vd0 = tc::smem_desc(ptx::smem_addr(v_half), kTile * 128, 1024, tc::kSwizzle128);
      const uint64_t pd0 = tc::smem_desc(ptx::smem_addr(p_at), 128, 16 * kTile, tc::kSwizzleNone);
      Walker walk(a, u0, u1, sh.b0, sh.ub0);
      int listed = 0;
      bool more = true;
      auto list = [&]() {  // one more segment, or the list's end
        const int n = listed++;
        if (n >= kSegRing) wait(sh.seg_empty[n % kSegRing], (n / kSegRing - 1) & 1);
        Segment s;
        more = walk.next(s);
        if (!more) s.tile1 = -1;
        if (lane == 0) sh.seg[n % kSegRing] = s;
        warp_arrive(sh.seg_full[n % kSegRing]);
      };
      Turns turns;
      uint32_t k = 0;
      for (int n_seg = 0;; ++n_seg) {
#pragma unroll 1
        while (more && listed < n_seg + kSegAhead) list();
        const Segment* seg = segment(n_seg);
        if (seg == nullptr) break;
        const int par = n_seg & 1;
        const int by_log2 = seg->by_log2, buf_log2 = seg->buf_log2, o_cols = seg->o_cols(), p_bytes = p_stride(buf_log2);
        const uint32_t io = tc::instr(D, 16 * seg->m, true, true);
        const int tiles = seg->tile1 - seg->tile0;
        if (n_seg >= 2) wait(sh.o_empty[par], ((n_seg >> 1) - 1) & 1);
#pragma unroll 1
        for (int i = 0; i < tiles; ++i, ++k) {
          const int buf = i & ((1 << buf_log2) - 1);
          const uint64_t vd = vd0 + (k & 1) * (L::kHalfBytes / 16);
          const uint64_t pd = pd0 + buf * (p_bytes / 16);
          const uint32_t dst = tmem + kOutAt + par * kAttnRows + (i & ((1 << by_log2) - 1)) * o_cols;
          const bool add = i >> by_log2 != 0;
          wait(sh.f_full[k & 1], (k >> 1) & 1);
          wait(sh.p_full[buf], turns.of(i, buf_log2));
          tc::fence_after();
          if (tc::elect()) {
#pragma unroll
            for (int j = 0; j < kTile / 16; ++j) tc::mma_f16(dst, vd + j * 128, pd + j * 16, io, add || j > 0);
            tc::commit(ptx::smem_addr(&sh.pv_done[buf]));
            tc::commit(ptx::smem_addr(&sh.f_empty[k & 1]));
            if (i + 1 == tiles) tc::commit(ptx::smem_addr(&sh.o_full[par]));
          }
          __syncwarp();
        }
        turns.pass(tiles, buf_log2);
        leave(n_seg);
      }
      Waiter drain;
      if (tc::elect()) tc::commit(ptx::smem_addr(&sh.done[1]));
      __syncwarp();
      drain(sh.done[1], 0);
      if (drain.dead()) wait.looks = 0;
    }
  }
  __syncwarp();
  if (wait.dead()) atomicOr(a.err, SPECDEC_DEV_ERR_TIMEOUT);
  __syncthreads();
  if (warp == kCopyWarp) tc::dealloc(tmem, kTmemCols);
}

}  // namespace specdec
