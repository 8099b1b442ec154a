// The tiled block-128 FP8 GEMM kernel (block_gemm.hip instantiates it).
//
// Structure: persistent workgroups, one per compute unit, each computing
// BM x BN output tiles; WM x WN waves own (BM / WM) x 64 outputs in 16 x 16
// fragments.  A step is one K block of 128: every A and B row of the tile brings
// 128 bytes into one of ST LDS stages by 16-byte direct-to-LDS buffer loads
// (rows XOR-swizzled in 16-byte chunks), and the scales of the step's rows come
// along.  The buffer descriptors end at the tile's last valid row, so rows past
// it read as zeros and cost no traffic.  Loads run ahead and continue into the
// next tile, whose first steps land while the finished tile is stored.  Tiles
// are worked out some rounds ahead and kept in an LDS ring, because the loop has
// no registers to do it in.
//
// Per fragment of a step the matrix cores sum the block's 128 products from
// zero into a temporary T, and the vector unit adds T f to the accumulator, f =
// sa[row] sb (a lane's four values share one row of A, and a wave's columns lie
// in one 128-block of B).  T is added up two fragments later, under the matrix
// instructions in between.  A step's last fragment row multiplies after the
// barrier that ends the step, while the next step's first fragments are read.
//
// FAST: E4M3 operands on V_MFMA_F32_16X16X128_F8F6F4, which sums a lane's eight
// neighbouring products aligned to the largest of them, 13 bits deep
// (measured: 1.5e-5 of the norm at K = 128, falling with K).  Otherwise the
// codes are widened to FP16 (exactly) and multiplied by
// V_MFMA_F32_16X16X32_F16 at half the rate, with full FP32 sums.
//
// What bounds it: the matrix cores, at the clock that they leave.  Contiguous
// groups, 65536 rows x 3072 x 4096: 770 to 800 us over several cards, 2.06 to
// 2.14 PFLOP/s; the matrix cores work 56 % of the cycles, the additions (half as many issue cycles as the matrix
// instructions) and the fragments' LDS reads fill most of the others, and the
// clock falls to 1.6 - 1.8 GHz of 2.4.  FP32 results of 65536 rows in 32 K groups,
// 4096 x 1536, through FP16: 845 to 910 us, 0.91 to 0.98 PFLOP/s.
// Measured against it (the contiguous case unless said): 32 x 32 fragments in
// the same form 5 % slower; row / 8 swizzles as for 32-row fragments 3 %; loads
// spread over the whole step 1 to 4 %; two workgroups a compute unit with two
// small stages, wave priorities, additions three fragments later, blocks of 4 or
// 16 m-tiles: 0 to 2 % slower.
#pragma once

#include "block_gemm.hpp"

namespace hq {
namespace blk {

__device__ __forceinline__ uint32_t ufirst(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t ufirst64(int64_t v) {
  const uint64_t u = (uint64_t)v;
  return (int64_t)(((uint64_t)ufirst((uint32_t)(u >> 32)) << 32) | ufirst((uint32_t)u));
}

// A pointer that is the same in every lane, which the compiler cannot prove.
template <class T>
__device__ __forceinline__ const T* uniform(const T* p) {
  return reinterpret_cast<const T*>(ufirst64((int64_t)(uintptr_t)p));
}

// XOR swizzles of the eight 16-byte chunks of a 128-byte LDS row.  Two rows
// cover the 64 banks, so the rows of one parity that a 16-lane group of a
// fragment read touches need different slots: A's fragments are 16 rows in
// order, B's take rows 8 a + 4 e + b (a, b < 4; below).  With the swizzle that
// suits 32-row fragments, (row ^ row / 8) % 8, half of the LDS cycles were
// conflicts.
__device__ __forceinline__ int swz_a(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int swz_b(int row) { return ((row >> 2) & 6) | ((row >> 1) & 1); }

// Raw buffer descriptor over [base, base + bytes).  A tile's operands take
// less than 2^31 bytes, so an offset with bit 31 set lies outside.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

// Direct-to-LDS buffer loads of 16 / 4 bytes a lane (zeros when out of range)
// at voff + soff: lane j's result lands at LDS address lds + j * size.  In
// inline assembly, so that the compiler adds no waits of its own; the kernel
// waits on the vector-memory counter and a barrier before a stage is read.  m0
// is set inside each statement and used by nothing else; the load needs one
// wait state after that, which the compiler does not add inside a statement.
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               ::"v"(voff), "s"(r), "s"(soff), "s"(lds) : "memory");
}
// The same for bytes that one workgroup reads once (non-temporal policy).
__device__ __forceinline__ void dma16nt(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen nt lds"
               ::"v"(voff), "s"(r), "s"(soff), "s"(lds) : "memory");
}
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dword %0, %1, %2 offen lds"
               ::"v"(voff), "s"(r), "s"(soff), "s"(lds) : "memory");
}

template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Workgroup barrier without a fence: the waits above order the LDS traffic.
__device__ __forceinline__ void bar() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
}

template <int BM_, int BN_, int WM_, int WN_, int ST_, bool FAST_>
struct Cfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, ST = ST_;
  static constexpr bool FAST = FAST_;
  static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int WTM = BM / WM, WTN = BN / WN, FI = WTM / 16, FJ = WTN / 16;
  static constexpr int AL = BM / 8 / WAVES, BL = BN / 8 / WAVES;   // 16-byte loads a thread, per step
  static constexpr int STAGE = (BM + BN) * 128;
  static constexpr int NB = BN / 128;
  // Scales.  GROUPED: four steps' scales travel together, 16 bytes a row (one
  // cache line touched per row and load), into one of two buffers; this needs
  // four K blocks in a row of the operand.  Otherwise each step brings its own
  // dword per row.
  static constexpr bool GROUPED = ST == 2;
  // Two stages: they are refilled in halves (HALF below).
  static constexpr bool HALF = ST == 2;
  static constexpr int SBUF = GROUPED ? BM * 16 + 1024 : BM * 4 + 256;
  static constexpr int SBUFS = GROUPED ? 2 : ST;
  static constexpr int SMEM = ST * STAGE + SBUFS * SBUF;
  static constexpr int SW = BM / 64;              // waves that load A's scales; wave SW loads B's
  static_assert(WTM % 32 == 0 && WTN == 64 && BN % 128 == 0, "wave tiles");
  static_assert(AL >= 1 && BL >= 1 && BM / 8 % WAVES == 0 && BN / 8 % WAVES == 0, "whole loads");
  static_assert(BM % 64 == 0 && SW + 1 <= WAVES, "scale loads");
  static_assert(!HALF || (WTM == 16 * WAVES && FI == 8), "a load of A covers half of the fragment rows of one row of waves");
};

struct Table {
  int end[kMaxGroups];     // rows (or K) where group g ends
  int tiles[kMaxGroups];   // inclusive count of m-tiles (grouped row forms)
};

// Where a tile sits (uniform).
struct Tile {
  int g, slice, nk, kb0;
  int64_t row0, row_end, n0;
};
// Its operands from row row0 / column n0 on, and their extents in bytes.
struct Operands {
  const uint8_t *a, *b;
  const float *sa, *sb;
  uint32_t a_bytes, b_bytes, sa_bytes, sb_bytes;
};

// The next tiles of a workgroup, by round, kept in LDS: the loads look them up
// in the middle of a K loop, where there are no registers to work them out.
struct Upcoming {
  Tile t;
  Operands o;
};
constexpr int kRing = 8;

// Tiles are numbered in blocks of 8 m-tiles x all n-tiles, n-major inside a
// block, so that the tiles an XCD's workgroups run side by side share operand
// rows; K slices and K groups are outermost.
struct Order {
  int mt_total;            // m-tiles (all groups; of one group in the K form)
  int mt_per;              // m-tiles of a group (uniform rows)
  int nt;
  int total;
};

template <class C>
__device__ __forceinline__ Order make_order(const BlockGemmArgs& p, Table& t) {
  Order o;
  o.nt = (int)((p.n + C::BN - 1) / C::BN);
  o.mt_per = 0;
  if (p.form == kContiguous || p.form == kMasked) {
    if (p.form == kContiguous) {
      load_clamped_ends<C::THREADS>(t.end, p.group_end, p.groups, p.rows);
    } else {
      for (int g = threadIdx.x; g < p.groups; g += C::THREADS) {
        const int64_t v = p.counts[g], c = v < 0 ? 0 : (v > p.slot_rows ? p.slot_rows : v);
        t.end[g] = (int)(g * p.slot_rows + c);
      }
      __syncthreads();
    }
    for (int g = threadIdx.x; g < p.groups; g += C::THREADS) {
      const int64_t s = p.form == kMasked ? g * p.slot_rows : (g > 0 ? t.end[g - 1] : 0);
      t.tiles[g] = (int)((t.end[g] - s + C::BM - 1) / C::BM);
    }
    __syncthreads();
    o.mt_total = block_scan_1024<C::THREADS>(t.tiles, p.groups, OpAdd(), 0);
    o.total = o.mt_total * o.nt;
  } else if (p.form == kGroupK) {
    load_clamped_ends<C::THREADS>(t.end, p.group_end, p.groups, p.k);
    o.mt_total = (int)((p.rows + C::BM - 1) / C::BM);
    o.total = o.mt_total * o.nt * p.groups;
  } else {
    o.mt_per = (int)((p.slot_rows + C::BM - 1) / C::BM);
    o.mt_total = o.mt_per * p.groups;
    o.total = o.mt_total * o.nt * p.slices;
  }
  o.mt_total = (int)ufirst((uint32_t)o.mt_total);      // uniform, which the compiler cannot see in LDS values
  o.total = (int)ufirst((uint32_t)o.total);
  return o;
}

template <class C>
__device__ __forceinline__ Tile make_tile(const BlockGemmArgs& p, const Table& t, const Order& o, int id) {
  Tile tl;
  const int plane = o.mt_total * o.nt;
  const int outer = id / plane;
  id -= outer * plane;
  const int blk = id / (8 * o.nt), rem = id - blk * 8 * o.nt;
  const int left = o.mt_total - blk * 8, mb = left < 8 ? left : 8;
  const int nt = rem / mb, mt = blk * 8 + (rem - nt * mb);
  int g = 0, k0 = 0, k1 = p.nkb;
  int64_t row0, row_end;
  tl.slice = 0;
  if (p.form == kUniform) {
    g = mt / o.mt_per;
    row0 = g * p.slot_rows + (int64_t)(mt - g * o.mt_per) * C::BM;
    row_end = (g + 1) * p.slot_rows;
    tl.slice = (int)ufirst((uint32_t)outer);
    k0 = p.nkb * outer / p.slices;               // nkb is below 2^16, slices at most 16
    k1 = p.nkb * (outer + 1) / p.slices;
  } else if (p.form == kGroupK) {
    g = outer;
    row0 = (int64_t)mt * C::BM;
    row_end = p.rows;
    k0 = (g > 0 ? t.end[g - 1] : 0) / 128;
    k1 = t.end[g] / 128;
  } else {
    int lo = 0, hi = p.groups - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (t.tiles[mid] > mt) hi = mid;
      else lo = mid + 1;
    }
    g = lo;
    const int64_t s = p.form == kMasked ? g * p.slot_rows : (g > 0 ? t.end[g - 1] : 0);
    row0 = s + (int64_t)(mt - (g > 0 ? t.tiles[g - 1] : 0)) * C::BM;
    row_end = t.end[g];
  }
  tl.g = (int)ufirst((uint32_t)g);
  tl.row0 = ufirst64(row0);
  row_end = row0 + C::BM < row_end ? row0 + C::BM : row_end;
  tl.row_end = ufirst64(row_end);
  tl.n0 = ufirst64((int64_t)nt * C::BN);
  tl.kb0 = (int)ufirst((uint32_t)k0);
  tl.nk = (int)ufirst((uint32_t)(k1 - k0));
  return tl;
}

// An empty K range becomes one step on empty descriptors: zeros.
template <class C>
__device__ __forceinline__ Operands operands(const BlockGemmArgs& p, const Tile& t) {
  Operands o;
  const int64_t g = p.form == kGroupK ? 0 : t.g;
  const int64_t nb0 = t.n0 / 128;
  o.a = uniform(p.a + t.row0 * p.k);
  o.b = uniform(p.b + (g * p.n + t.n0) * p.k);
  o.sa = uniform(p.sa + t.row0 * p.nkb);
  o.sb = uniform(p.sb + (g * p.nnb + nb0) * p.nkb);
  const bool any = t.nk > 0;
  const uint32_t k = (uint32_t)p.k, sk = (uint32_t)p.nkb * 4;
  const uint32_t m = any ? (uint32_t)(t.row_end - t.row0) : 0;
  const uint32_t n = any ? (uint32_t)(p.n - t.n0 < C::BN ? p.n - t.n0 : C::BN) : 0;
  o.a_bytes = ufirst(m * k);
  o.b_bytes = ufirst(n * k);
  o.sa_bytes = ufirst(m * sk);
  o.sb_bytes = ufirst((n + 127) / 128 * sk);
  return o;
}

// OUT: BlockOut of the stores (a K split stores FP32 partials).  POL: BlockPolicy.
template <class C, int OUT, int POL>
__global__ __launch_bounds__(C::THREADS, 2) void block_gemm_tiled(BlockGemmArgs p) {
  constexpr int FI = C::FI, FJ = C::FJ, ST = C::ST, AL = C::AL, BL = C::BL;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ Table table;
  __shared__ Upcoming ring[kRing];
  const Order ord = make_order<C>(p, table);
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = (int)ufirst((uint32_t)(tid >> 6));
  const int wm = w / C::WN, wn = w % C::WN;

  // XCD-aware order: workgroup b runs on XCD b % 8.  A launch over one plane
  // of uniform tiles gives each XCD a contiguous eighth of them; other forms
  // give each XCD a contiguous run of every round, odd rounds backwards.
  const int nx = gridDim.x >= 8 ? 8 : 1, per = gridDim.x / nx;
  if ((int)blockIdx.x >= per * nx) return;
  const int x = blockIdx.x % nx, ci = blockIdx.x / nx;
  const bool eighths = p.form == kUniform && p.groups == 1 && p.slices == 1;
  auto eighth = [&](int i) { return nx == 8 ? (int)((int64_t)ord.total * i >> 3) : ord.total * i; };
  const int first = eighths ? eighth(x) + ci : 0;
  const int last = eighths ? eighth(x + 1) : ord.total;
  auto tile_at = [&](int round) -> int {
    if (eighths) return first + round * per;
    const int slot = x * per + ci, stride = per * nx;
    return round * stride + ((round & 1) ? stride - 1 - slot : slot);
  };
  if (tile_at(0) >= last) {
    // a backwards second round may still hold a tile for this workgroup only
    // if the first one was full: then tile_at(0) < last
    return;
  }

  // Load offsets, the same for every tile and step: load i of wave w fills
  // LDS rows (i WAVES + w) 8 .. + 7, lane j the chunk that belongs at slot
  // j % 8 of row j / 8.  The swizzles do not depend on i (WAVES is a multiple of
  // 4), so one offset serves all loads of an operand and the descriptor moves.
  uint32_t offa, offb;               // bit 31 drops a load
  uint32_t dropa, dropb;             // its value for chunks past the last, partial K block's end
  {
    const uint32_t krem = (uint32_t)p.k & 127, row = w * 8 + (lane >> 3);
    const uint32_t ca = ((lane & 7) ^ swz_a(row)) * 16, cb = ((lane & 7) ^ swz_b(row)) * 16;
    offa = row * (uint32_t)p.k + ca;
    offb = row * (uint32_t)p.k + cb;
    dropa = krem != 0 && ca >= krem ? 0x80000000u : 0u;
    dropb = krem != 0 && cb >= krem ? 0x80000000u : 0u;
  }
  static_assert(C::WAVES % 4 == 0, "the swizzles' period");
  const uint32_t hop = (uint32_t)p.k * (C::WAVES * 8);      // bytes from one load's rows to the next one's
  const uint32_t lds0 = ufirst((uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)smem);

  // Every wave writes the same values and reads its own; it runs at most a
  // step ahead of the others, so a slot is not reused while it is needed.
  auto plan = [&](int round) {
    Upcoming u;
    const int id = tile_at(round);
    if (id < last) {
      u.t = make_tile<C>(p, table, ord, id);
      u.o = operands<C>(p, u.t);
    } else {                 // nothing left: steps load zeros from empty descriptors
      u.t = Tile{};
      u.t.nk = 0x7FFFFFFF;
      u.o = Operands{};
    }
    if (lane == 0) ring[round % kRing] = u;
  };
  // With one step a tile, the loads' cursor ends a step of round r at round r +
  // ST: the rounds up to there are planned.
  static_assert(ST + 2 <= kRing, "tiles in flight");
#pragma unroll 1
  for (int r = 0; r <= ST; ++r) plan(r);
  auto upcoming = [&](int round) -> Operands {
    const Operands& v = ring[round % kRing].o;
    Operands o;
    o.a = uniform(v.a);
    o.b = uniform(v.b);
    o.sa = uniform(v.sa);
    o.sb = uniform(v.sb);
    o.a_bytes = ufirst(v.a_bytes);
    o.b_bytes = ufirst(v.b_bytes);
    o.sa_bytes = ufirst(v.sa_bytes);
    o.sb_bytes = ufirst(v.sb_bytes);
    return o;
  };
  auto tile_of = [&](int round) -> Tile {
    const Tile& v = ring[round % kRing].t;
    Tile t;
    t.g = (int)ufirst((uint32_t)v.g);
    t.slice = (int)ufirst((uint32_t)v.slice);
    t.nk = (int)ufirst((uint32_t)v.nk);
    t.kb0 = (int)ufirst((uint32_t)v.kb0);
    t.row0 = ufirst64(v.row0);
    t.row_end = ufirst64(v.row_end);
    t.n0 = ufirst64(v.n0);
    return t;
  };

  // ---------------------------------------------------------------- loads
  int lround = 0, lk = 0, lstep = 0, lgroup = 0;   // load cursor: tile round, step in it, stage, scale buffer
  int lkb0, lnk;                                   // that tile's first K block and its steps
  Operands lo = upcoming(0);
  {
    const Tile t = tile_of(0);
    lkb0 = t.kb0;
    lnk = t.nk;
  }
  // issues part `part` of `parts` of the cursor's step's loads first .. first +
  // count - 1, B's and then A's (HALF: A's even ones, then its odd ones); bit 31
  // of an offset drops the load
  auto issue = [&](int part, int parts, int first, int count) {
    const int kb = lkb0 + lk;
    const uint32_t st = lds0 + (uint32_t)lstep * C::STAGE + (uint32_t)w * 1024;
    const uint32_t ko = (uint32_t)kb * 128;
    const bool tail = kb == p.nkb - 1;
    const uint32_t va = offa | (tail ? dropa : 0u), vb = offb | (tail ? dropb : 0u);
    // operand load i of the descriptor [base, base + bytes)
    auto load = [&](const uint8_t* base, uint32_t bytes, uint32_t v, int i, uint32_t lds, auto nt) {
      const int rest = (int)bytes - (int)(i * hop);         // signed: a scalar maximum
      const __amdgpu_buffer_rsrc_t r = rsrc(base + i * hop, (uint32_t)(rest > 0 ? rest : 0));
      if constexpr (decltype(nt)::value) dma16nt(r, v, ko, lds + i * C::WAVES * 1024);
      else dma16(r, v, ko, lds + i * C::WAVES * 1024);
    };
#pragma unroll
    for (int l = 0; l < AL + BL; ++l) {
      if (l < first || l >= first + count || part != (l - first) * parts / count) continue;
      const int i = l < BL ? l : !C::HALF ? l - BL : (l - BL) * 2 < AL ? (l - BL) * 2 : (l - BL) * 2 - AL + 1;
      if (l < BL) load(lo.b, lo.b_bytes, vb, i, st + C::BM * 128, std::bool_constant<POL == kPolStreamAll>());
      else load(lo.a, lo.a_bytes, va, i, st, std::false_type());
    }
  };
  // Scales: waves 0 .. SW - 1 bring 64 rows of A each, wave SW the B blocks'.
  auto issue_scales = [&]() {
    if (w > C::SW || (C::GROUPED && (lk & 3) != 0)) return;
    const int kb = lkb0 + lk;
    const bool isb = w == C::SW;
    const __amdgpu_buffer_rsrc_t r = isb ? rsrc(lo.sb, lo.sb_bytes) : rsrc(lo.sa, lo.sa_bytes);
    const uint32_t row = isb ? lane : w * 64 + lane;
    const uint32_t v = row * (uint32_t)p.nkb * 4 | (isb && lane >= C::NB ? 0x80000000u : 0u);
    const uint32_t sb = ufirst(lds0 + ST * C::STAGE + (uint32_t)(C::GROUPED ? lgroup : lstep) * C::SBUF);
    if constexpr (C::GROUPED)      // the last steps' four start early enough to end with the row
      dma16(r, v, (uint32_t)(kb < p.nkb - 4 ? kb : p.nkb - 4) * 4, sb + (isb ? C::BM * 16 : w * 1024));
    else
      dma4(r, v, (uint32_t)kb * 4, sb + (isb ? C::BM * 4 : w * 256));
  };
  auto advance = [&]() {
    lstep = lstep + 1 == ST ? 0 : lstep + 1;
    ++lk;
    if (C::GROUPED && (lk & 3) == 0) lgroup ^= 1;
    if (lk >= lnk) {
      if (C::GROUPED && (lk & 3) != 0) lgroup ^= 1;
      lk = 0;
      ++lround;
      lo = upcoming(lround);
      lkb0 = (int)ufirst((uint32_t)ring[lround % kRing].t.kb0);
      lnk = (int)ufirst((uint32_t)ring[lround % kRing].t.nk);
    }
  };
  auto issue_all = [&]() {
    issue_scales();
#pragma unroll
    for (int s = 0; s < AL + BL; ++s) issue(s, AL + BL, 0, AL + BL);
  };
  // vector-memory operations of a step per wave, where that is the same for every step
  constexpr int kOps = AL + BL;
  // HALF: a stage is refilled in two halves.  Its early loads are B and the A
  // rows of the first half of the fragment rows, its late ones the rest of A.
  // When a step has read its first half (B's fragments stay in registers) a
  // barrier in its middle frees that half, and the early loads of the step after
  // next go there; the late ones follow at the start of the next step.  Each
  // half has a step and a half to land: it is waited for where it is first read,
  // at the end of the step before (early) or in the middle of its own (late),
  // with one younger half step of each kind, kOps operations, in flight.
  constexpr int kEarly = BL + AL / 2, kLate = AL - AL / 2;
  auto issue_early = [&]() {
    issue_scales();
#pragma unroll
    for (int s = 0; s < kEarly; ++s) issue(s, kEarly, 0, kEarly);
  };
  if constexpr (C::HALF) {
    issue_early();
#pragma unroll
    for (int s = 0; s < kLate; ++s) issue(s, kLate, kEarly, kLate);
    advance();
    issue_early();
  } else {
#pragma unroll 1
    for (int s = 0; s < ST - 1; ++s) {
      issue_all();
      advance();
    }
  }
  // waits until the next step's loads have landed: the operations of the ST - 2
  // steps after it may stay in flight.  Memory
  // operations retire in the order of issue, so later stores only make the
  // wait stricter.
  auto land = [&]() {
    if constexpr (C::HALF) wait_vm<kOps>();      // scales and stores among them make the wait stricter
    else if (w <= C::SW) wait_vm<(ST - 2) * (kOps + 1)>();
    else wait_vm<(ST - 2) * kOps>();
    bar();
  };
  land();

  // ---------------------------------------------------------------- compute
  // Fragments of 16 rows: lane l holds row l % 16, chunks q and 4 + q (q = l /
  // 16) of its 128 codes.  A's fragment i starts at the wave's LDS row 16 i.
  // B's fragments come in pairs over 32 columns, interleaved by fours, so that
  // the accumulators of a pair are eight neighbouring columns of a lane:
  // row x of fragment j is column 32 (j / 2) + 8 (x / 4) + 4 (j % 2) + x % 4.
  const int x16 = lane & 15, q = lane >> 4;
  const uint32_t xa = (uint32_t)(x16 * 128 + ((q ^ swz_a(x16)) << 4));       // byte offset of chunk q; ^ 64: of chunk 4 + q
  const uint32_t xb = (uint32_t)((8 * (x16 >> 2) + (x16 & 3)) * 128 + ((q ^ swz_b(8 * (x16 >> 2) + (x16 & 3))) << 4));
  // A fragment's 32 codes of a lane; whole vectors throughout, so that they
  // stay in consecutive registers across the loop.
  auto rd = [](const uint8_t* at, uint32_t xo) -> v8i {
    const v4i lo4 = *reinterpret_cast<const v4i*>(at + xo), hi4 = *reinterpret_cast<const v4i*>(at + (xo ^ 64u));
    return __builtin_shufflevector(lo4, hi4, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  auto rd_a = [&](const uint8_t* stage_at, int i) { return rd(stage_at + wm * C::WTM * 128 + i * 2048, xa); };
  auto rd_b = [&](const uint8_t* stage_at, int j) {
    return rd(stage_at + C::BM * 128 + wn * C::WTN * 128 + (j >> 1) * 4096 + (j & 1) * 512, xb);
  };

  // Steps overlap: the last fragment row of a step multiplies after the barrier
  // that ends it (head), while the next step's first fragments are read into the
  // registers that it frees; the other rows (body) follow, with the loads.  So
  // the matrix cores have work while the first reads of a step are under way,
  // and every fragment of a step has been read when the barrier frees its stage.
  v4f acc[FI][FJ];
  int stage = 0, group = 0;
  constexpr int G = FI * FJ, GB = G - FJ;     // fragments of a step, of its body
  constexpr int LS = GB < AL + BL ? GB : AL + BL;     // load slots, from the body's first fragment on
  constexpr int kMid = FI / 2 - 1;            // HALF: the row before which a step's first half has been read
  auto issue_at = [&](int g) {                // the loads of the body's fragment g
    if constexpr (C::HALF) {
      if (g < kLate) issue(g, kLate, kEarly, kLate);
      else if (g >= kMid * FJ && g < kMid * FJ + kEarly) issue(g - kMid * FJ, kEarly, 0, kEarly);
    } else if (g < LS) {
      issue(g, LS, 0, AL + BL);
    }
  };
  auto fence = [&]() { __builtin_amdgcn_sched_barrier(0); };
  constexpr int D = C::FAST ? 1 : 2;
  v4f tm[D][FJ];                // FAST: fragment g's sum, added up two fragments later; else a row's, added during the next
  float f[FI], flast = 0.0f;    // the step's factors; the last row's, of the step before
  v8i ra[2];                    // A's fragments of this row and the next
  v8i rb[FJ];                   // B's
  v8h da[C::FAST ? 1 : 2][4], db[C::FAST ? 1 : FJ][4];     // widened
  auto add = [&](int i, int j, float fi) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      acc[i][j][r] = __builtin_fmaf(tm[C::FAST ? 0 : i & 1][j][r], fi, acc[i][j][r]);
  };
  auto widen1 = [](const v8i& r, int e) -> v8h { return decode_fp8x8((uint32_t)r[2 * e], (uint32_t)r[2 * e + 1]); };
  // the first fragments of the current stage's step
  auto read_first = [&]() {
    const uint8_t* base = smem + stage * C::STAGE;
    ra[0] = rd_a(base, 0);
#pragma unroll
    for (int j = 0; j < FJ; ++j) rb[j] = rd_b(base, j);
    if constexpr (!C::FAST) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        da[0][e] = widen1(ra[0], e);
#pragma unroll
        for (int j = 0; j < FJ; ++j) db[j][e] = widen1(rb[j], e);
      }
    }
  };
  // the factors of place k of tile t
  auto read_f = [&](const Tile& t, int k) {
    const int row = wm * C::WTM + x16, nb = wn * C::WTN / 128;
    const uint8_t* s = smem + ST * C::STAGE;
    float sbv, v[FI];
    if constexpr (C::GROUPED) {
      const int kb = t.kb0 + k, g0 = t.kb0 + (k & ~3);
      s += group * C::SBUF + (kb - (g0 < p.nkb - 4 ? g0 : p.nkb - 4)) * 4;
      sbv = *reinterpret_cast<const float*>(s + C::BM * 16 + nb * 16);
#pragma unroll
      for (int i = 0; i < FI; ++i) v[i] = *reinterpret_cast<const float*>(s + (row + 16 * i) * 16);
    } else {
      s += stage * C::SBUF;
      sbv = *reinterpret_cast<const float*>(s + C::BM * 4 + nb * 4);
#pragma unroll
      for (int i = 0; i < FI; ++i) v[i] = *reinterpret_cast<const float*>(s + (row + 16 * i) * 4);
    }
    // an empty K range: the codes read as zeros, the scales as anything
    const bool any = t.nk != 0;
#pragma unroll
    for (int i = 0; i < FI; ++i) f[i] = any ? v[i] * sbv : 0.0f;
  };
  // Row i of the step whose fragments are in registers.  next: base of the row
  // read for after it (row 0 of the next step for the last row, whose B
  // fragments are replaced too).
  auto row = [&](auto ic) {
    constexpr int i = decltype(ic)::value;
    constexpr bool kHead = i == FI - 1;
    const uint8_t* base = smem + stage * C::STAGE;
    if constexpr (C::FAST) {
      ra[(i + 1) & 1] = rd_a(base, kHead ? 0 : i + 1);
#pragma unroll
      for (int j = 0; j < FJ; ++j) {
        constexpr int kBack = 2;       // added up this many fragments later
        const int g = i * FJ + j;
        tm[0][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(rb[j], ra[i & 1], v4f{}, 0, 0, 0, 0, 0, 0);
        if (!kHead) issue_at(g);
        fence();
        if constexpr (kHead) rb[j] = rd_b(base, j);
        if (g >= kBack) add((g - kBack) / FJ, (g - kBack) % FJ, f[(g - kBack) / FJ]);
        else add(FI - 1, FJ - kBack + g, flast);
        fence();
      }
    } else {
      ra[0] = rd_a(base, kHead ? 0 : i + 1);
      if constexpr (kHead) {
#pragma unroll
        for (int j = 0; j < FJ; ++j) rb[j] = rd_b(base, j);
      }
      fence();
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int j = 0; j < FJ; ++j)
          tm[i & 1][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(db[j][e], da[i & 1][e], e == 0 ? v4f{} : tm[i & 1][j],
                                                                0, 0, 0);
        if (!kHead) issue_at(i * FJ + e);
        if (i > 0) add(i > 0 ? i - 1 : 0, e, f[i > 0 ? i - 1 : 0]);
        else add(FI - 1, e, flast);
        if (e > 0) {
          da[(i + 1) & 1][e - 1] = widen1(ra[0], e - 1);
          if constexpr (kHead) {
#pragma unroll
            for (int j = 0; j < FJ; ++j) db[j][e - 1] = widen1(rb[j], e - 1);
          }
        }
        fence();
      }
      da[(i + 1) & 1][3] = widen1(ra[0], 3);
      if constexpr (kHead) {
#pragma unroll
        for (int j = 0; j < FJ; ++j) db[j][3] = widen1(rb[j], 3);
      }
    }
  };
  // Keeps the sums ahead of what follows: the compiler would otherwise sink
  // them past the branches there and hold a temporary for every fragment.
  auto pin = [&]() {
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
      for (int j = 0; j < FJ; ++j) asm volatile("" : "+v"(acc[i][j]));
  };
  // HALF: the first half of the step's stage has been read, its second has landed
  auto middle = [&]() {
    advance();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    land();
    issue_scales();
  };
  auto body = [&](auto self, auto ic) -> void {
    constexpr int i = decltype(ic)::value;
    if constexpr (i < FI - 1) {
      if constexpr (C::HALF && i == kMid) {
        pin();
        middle();
      }
      row(ic);
      self(self, std::integral_constant<int, i + 1>());
    }
  };
  static_assert(FI >= 2 && FI % 2 == 0 && FJ == 4, "A's two fragment buffers alternate across steps");
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
      for (int j = 0; j < FJ; ++j) acc[i][j] = v4f{};
  };

  int round = 0;
  bool have = false;            // the current step's first fragments are in registers
  Tile t = tile_of(0);
  clear();
  for (;;) {
    const int nk = t.nk > 0 ? t.nk : 1;
    // A wave whose rows all lie past the tile's last one only loads its share.
    const bool active = t.row0 + wm * C::WTM < t.row_end;
    auto next = [&](int k) {     // ends step k: the next step's loads have landed
      if constexpr (!C::HALF) advance();
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");      // the stage has been read
      land();
      stage = stage + 1 == ST ? 0 : stage + 1;
      if (k + 1 == nk || (C::GROUPED && (k & 3) == 3)) group ^= 1;
    };
    if (active) {
      if (!have) read_first();
      flast = 0.0f;
#pragma unroll
      for (int j = 0; j < FJ; ++j) tm[D - 1][j] = v4f{};
      for (int k = 0; k < nk; ++k) {
        if constexpr (!C::HALF) issue_scales();
        read_f(t, k);
        body(body, std::integral_constant<int, 0>());
        pin();
        next(k);
        row(std::integral_constant<int, FI - 1>());
        pin();
        flast = f[FI - 1];
      }
      if constexpr (C::FAST) {
        add(FI - 1, FJ - 2, flast);
        add(FI - 1, FJ - 1, flast);
      } else {
#pragma unroll
        for (int j = 0; j < FJ; ++j) add(FI - 1, j, flast);
      }
    } else {
      for (int k = 0; k < nk; ++k) {
        if constexpr (!C::HALF) issue_scales();
#pragma unroll
        for (int g = 0; g < GB; ++g) {
          if (C::HALF && g == kMid * FJ) middle();
          issue_at(g);
        }
        next(k);
      }
    }
    have = active;

    // ------------------------------------------------------------ epilogue
    // Through LDS, so that a store writes whole lines: a lane's accumulators
    // are eight columns of one row (a pair of fragments holds columns 32 jp +
    // 8 q + 0 .. 7), and stored from there each 16 lanes would touch 16 lines.  A
    // wave puts kRows fragment rows at a time into its share of the stage that
    // the next step's loads will fill (all of it has been read) and stores them
    // row by row, 16 bytes a lane.
    if (active) {
      constexpr int ES = OUT == kOutBf16 || OUT == kOutF16 ? 2 : 4;
      // HALF: the late loads' part of the stage; a row of waves has its own
      constexpr int kShare = C::HALF ? C::WTM / 2 * 128 / C::WN : C::STAGE / C::WAVES;
      constexpr int kPairs = 16 * C::WTN * ES <= kShare ? FJ / 2 : 1;     // column pairs of fragments at a time
      constexpr int RB = kPairs * 32 * ES, CH = RB / 16;       // bytes and 16-byte chunks of their rows
      constexpr int kFit = kShare / (16 * RB), kRows = kFit >= 4 && FI % 4 == 0 ? 4 : (kFit >= 2 ? 2 : 1);
      static_assert(kFit >= 1 && FI % kRows == 0, "a fragment row fits a wave's share of a stage");
      int ln = lane;                       // opaque: nothing below is kept through the K loop
      asm volatile("" : "+v"(ln));
      const int x16 = ln & 15, q = ln >> 4;
      uint8_t* mine = smem + lstep * C::STAGE +
                      (C::HALF ? wm * C::WTM * 128 + C::WTM / 2 * 128 + wn * kShare : w * kShare);
      auto slot = [](int row, int ch) { return row * RB + ((ch ^ (CH == 8 ? (row >> 1) & 7 : row & 15)) << 4); };
      const int64_t orow = (p.form == kGroupK ? (int64_t)t.g * p.rows : 0) + (int64_t)t.slice * p.rows;
      const int lrow = ln / CH, ch = ln % CH;                  // a store instruction: 64 / CH rows
      const int64_t row = t.row0 + wm * C::WTM + lrow, n = t.n0 + wn * C::WTN + ch * (16 / ES);
      uint8_t* dst = static_cast<uint8_t*>(p.out) + ((orow + row) * p.ldo + n) * ES;
#pragma unroll
      for (int b = 0; b < FI / kRows * (FJ / 2 / kPairs); ++b) {
        const int i0 = b / (FJ / 2 / kPairs) * kRows, j0 = b % (FJ / 2 / kPairs) * kPairs;
        const int64_t left = n + j0 * 32 < p.n ? t.row_end - row : 0;      // rows of the lane's column from here on
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
          for (int jp = 0; jp < kPairs; ++jp) {
            const v4f lo4 = acc[i0 + i][2 * (j0 + jp)], hi4 = acc[i0 + i][2 * (j0 + jp) + 1];
            if constexpr (ES == 2) {
              constexpr bool F16 = OUT == kOutF16;
              *reinterpret_cast<uint4*>(mine + slot(16 * i + x16, 4 * jp + q)) =
                  make_uint4(pack_half2<F16>(lo4[0], lo4[1]), pack_half2<F16>(lo4[2], lo4[3]),
                             pack_half2<F16>(hi4[0], hi4[1]), pack_half2<F16>(hi4[2], hi4[3]));
            } else {
              *reinterpret_cast<v4f*>(mine + slot(16 * i + x16, 8 * jp + 2 * q)) = lo4;
              *reinterpret_cast<v4f*>(mine + slot(16 * i + x16, 8 * jp + 2 * q + 1)) = hi4;
            }
          }
        fence();
#pragma unroll
        for (int c = 0; c < 16 * kRows / (64 / CH); ++c) {
          const int r = 16 * i0 + c * (64 / CH);               // the instruction's first row in the wave tile
          v4f v = *reinterpret_cast<const v4f*>(mine + slot(c * (64 / CH) + lrow, ch));
          if (r < left) {
            v4f* d = reinterpret_cast<v4f*>(dst + (r * p.ldo + j0 * 32) * ES);
            if constexpr (OUT == kOutF32Add) v = *d + v;
            if constexpr (POL != kPolKeep) __builtin_nontemporal_store(v, d);
            else *d = v;
          }
        }
        fence();
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    bar();                // every wave is done with that stage
    if (tile_at(++round) >= last) break;
    plan(round + ST);
    t = tile_of(round);
    clear();
  }
  wait_vm<0>();       // no load may land in LDS after the workgroup has ended
}

}  // namespace blk
}  // namespace hq
