// The tiled 16-bit GEMM kernel (half_plan.hpp picks the shape; half_nt.hip, half_nn.hip
// and half_tn.hip instantiate it).
//
// out = sum over k of a b, per tile in FP32 on the matrix cores (products of 16-bit
// values are exact there), rounded once.  Persistent workgroups of 4 waves (2 for
// 32x64), one a compute unit.  With 256x256 tiles a wave has 128x128 sums in half
// of its registers and reads 16 fragments for 64 products, so that LDS (128 bytes a
// cycle) needs half of the matrix cores' time; with 128x128 tiles all of it, which
// those pay with 0.37 of a large tile's time for a quarter of its work.  Operands
// go straight to LDS, 64 K values a step, two steps ahead (large tiles) to nine.
// 65536 rows of 32 experts, 4096 x 1536: 673 to 711 us by card, 1.16 to 1.23 PFLOP/s (a
// library's dense product of this size 687 us), b transposed 683 to 718 us, the weights'
// sums over rows (both operands read transposed from LDS, 805 MB of results) 713 to
// 740 us.  Bound: the matrix cores are busy for 55 to 61 % of the cycles at the 1.9 GHz
// that power leaves (all operands zero: 614 us of 675); the rest of the cycles is a
// tile's fill and epilogue, with one workgroup a unit to cover them.
// Accumulated FP32 results are the slow ones: each share of a tile is loaded, waited
// for, added to and stored before the next one's load, a chain of trips to memory:
// 1216 us where plain FP32 results take 758, sums over rows 1046 and 713, and 303 and
// 88 where a group has 128 rows (32 groups, 2048 x 1536).
// Against it: 32x32x16 fragments 3-5 % slower (2.5 % faster on zeros), steps of 32 K
// values in four stages 777 us, loads bunched at a half's start 4 % slower.
#pragma once

#include <utility>

#include "block_gemm.hpp"
#include "half_internal.hpp"
#include "half_math.hpp"
#include "tile_util.hpp"

namespace hq {
namespace half {

using namespace blk;

// acc += a b^T for fragments of 16 x 32 values (BF16 or FP16 bits), in place: as
// builtins the compiler gives results other registers than the sums they
// continue and copies sums around them, 300 moves in a step of 128 products.  The
// compiler puts no wait states before these: the kernel has them where sums are
// cleared and read, and fragments come from LDS loads, which it waits for.
template <bool F16, bool AGPR>
__device__ __forceinline__ void mfma(v4f& acc, v4i a, v4i b) {
  if constexpr (AGPR) {
    if constexpr (F16) asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
    else asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
  } else {
    if constexpr (F16) asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+v"(acc) : "v"(a), "v"(b));
    else asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+v"(acc) : "v"(a), "v"(b));
  }
}

// f(0), .., f(N - 1) with the numbers as constants (the compiler gives up
// unrolling loops of this size).
template <class F, int... I>
__device__ __forceinline__ void each_of(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>()), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F f) {
  each_of(f, std::make_integer_sequence<int, N>());
}

template <int BM_, int BN_, int WM_, int WN_, int ST_>
struct Cfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, ST = ST_;
  static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int WTM = BM / WM, WTN = BN / WN, FI = WTM / 16, FJ = WTN / 16;
  static constexpr int AL = BM / 8 / WAVES, BL = BN / 8 / WAVES;   // loads a wave, per step of 64 K values
  static constexpr int STAGE = (BM + BN) * 128;
  static constexpr bool BIG = FI * FJ >= 64;        // sums that take half of the register file
  // the epilogue's share of a wave: 16 rows of at most 256 bytes, padded
  static constexpr int EROW = WTN * 2 < 256 ? WTN * 2 : 256, ESTRIDE = EROW + 16, ESHARE = 16 * ESTRIDE;
  static constexpr int SMEM = ST * STAGE + WAVES * ESHARE;
  static_assert(BM / 8 % WAVES == 0 && BN / 8 % WAVES == 0 && AL >= 1 && BL >= 1, "whole loads");
  static_assert(WAVES % 2 == 0, "the row swizzle's period");
  static_assert((AL + BL) * (ST - 1) <= 63, "the vector-memory counter");
};

struct Table {
  int end[kMaxGroups];     // rows where group g ends
  int tiles[kMaxGroups];   // row forms: inclusive count of m-tiles; else: the groups, longest first
};
constexpr int kSortedGroups = 128;

// Where a tile sits (uniform).
struct Tile {
  int g, nk;
  int64_t row0, row_end, n0;
};
constexpr int kRing = 16;

// LDS layouts of an operand's step.  ROW: 128-byte rows, 16-byte chunks
// XOR-swizzled.  COL (T): 64 rows of W columns, 32-byte pieces XOR-swizzled.
__device__ __forceinline__ int swz_row(int row) { return (row >> 1) & 7; }
template <int W>
__device__ __forceinline__ int swz_col(int krow) {
  return ((krow & 3) | ((krow >> 3) & 1) << 2) & (W / 16 < 8 ? W / 16 - 1 : 7);
}

// Source offset (bytes) of lane `lane` of the wave-load number `ld`.
template <bool T, int W>
__device__ __forceinline__ uint32_t load_offset(int ld, int lane, uint32_t pitch) {
  if constexpr (!T) {
    const int row = ld * 8 + (lane >> 3);
    return (uint32_t)row * pitch + (uint32_t)(((lane & 7) ^ swz_row(row)) << 4);
  } else {
    constexpr int CH = W / 8;                       // 16-byte chunks of a K row
    const int krow = ld * (64 / CH) + lane / CH, c = lane % CH;
    return (uint32_t)krow * pitch + (uint32_t)((((c >> 1) ^ swz_col<W>(krow)) << 1 | (c & 1)) << 4);
  }
}

// Reads of the fragments (16 rows or columns x 32 K values) of a wave: lane
// (x, q) holds K values 8 q .. + 7 of half `ks` of the step, of row or column x.
template <bool T, int W, int F>
struct Frags {
  static constexpr int N = T ? F : 2;
  uint32_t off[N], at[N];       // the lane's offsets in a stage, and in the one that is read; ROW: by half, COL: by fragment
  __device__ __forceinline__ void init(int lane, int wave_base) {
    const int x = lane & 15, q = lane >> 4, krow = 8 * q + (x >> 2);
#pragma unroll
    for (int i = 0; i < N; ++i)
      off[i] = !T ? (uint32_t)((wave_base + x) * 128 + (((4 * i + q) ^ swz_row(x)) << 4))
                  : (uint32_t)(krow * 2 * W + (((wave_base / 16 + i) ^ swz_col<W>(krow)) << 5) + 8 * (x & 3));
  }
  __device__ __forceinline__ void stage(uint32_t base, int ks) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (T || i == ks) at[i] = base + off[i];
  }
  __device__ __forceinline__ v4i read(int i, int ks) const {
    typedef __attribute__((address_space(3))) uint8_t lds8;
    if constexpr (!T) {
      const lds8* p = (const lds8*)(uintptr_t)at[ks];
      return *(const __attribute__((address_space(3))) v4i*)(p + i * 2048);
    } else {
      lds8* p = (lds8*)(uintptr_t)at[i] + ks * 64 * W;
      typedef __attribute__((address_space(3))) v4s lds4;
      const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)p);
      const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + 8 * W));
      typedef short v8s __attribute__((ext_vector_type(8)));
      return __builtin_bit_cast(v4i, (v8s)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

// AT / BT: the operand lies K-major outside (K rows of columns).
template <class C, bool AT, bool BT, bool F16>
__global__ __launch_bounds__(C::THREADS, 1) void half_gemm_tiled(HalfGemmArgs p) {
  constexpr int FI = C::FI, FJ = C::FJ, ST = C::ST, AL = C::AL, BL = C::BL;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ Table table;
  __shared__ Tile ring[kRing];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = (int)ufirst((uint32_t)(tid >> 6));
  const int wm = w / C::WN, wn = w % C::WN;

  // ---------------------------------------------------------------- tiles
  const int nt = (int)((p.n + C::BN - 1) / C::BN);
  int mt_total;
  if constexpr (AT) {
    load_clamped_ends<C::THREADS>(table.end, p.group_end, p.groups, p.k);
    mt_total = (int)((p.rows + C::BM - 1) / C::BM);
    // Workgroups take whole rounds of tiles, a group's after the other's: with the
    // longest first the rounds at the end, where they differ, are the short ones
    // (more groups than kSortedGroups come as they are: the search is quadratic).
    for (int g = tid; g < p.groups; g += C::THREADS) {
      int rank = g;
      if (p.groups <= kSortedGroups) {
        auto len = [&](int i) { return table.end[i] - (i > 0 ? table.end[i - 1] : 0); };
        const int mine = len(g);
        rank = 0;
        for (int i = 0; i < p.groups; ++i) rank += len(i) > mine || (len(i) == mine && i < g);
      }
      table.tiles[rank] = g;
    }
    __syncthreads();
  } else {
    if (p.form == kContiguous) {
      load_clamped_ends<C::THREADS>(table.end, p.group_end, p.groups, p.rows);
    } else {
      for (int g = tid; g < p.groups; g += C::THREADS) {
        const int64_t v = p.counts[g], c = v < 0 ? 0 : (v > p.slot_rows ? p.slot_rows : v);
        table.end[g] = (int)(g * p.slot_rows + c);
      }
      __syncthreads();
    }
    for (int g = tid; g < p.groups; g += C::THREADS) {
      const int64_t s = p.form == kMasked ? g * p.slot_rows : (g > 0 ? table.end[g - 1] : 0);
      table.tiles[g] = (int)((table.end[g] - s + C::BM - 1) / C::BM);
    }
    __syncthreads();
    mt_total = block_scan_1024<C::THREADS>(table.tiles, p.groups, OpAdd(), 0);
  }
  mt_total = (int)ufirst((uint32_t)mt_total);
  const int total = AT ? mt_total * nt * p.groups : mt_total * nt;

  // XCD-aware order: workgroup b runs on XCD b % 8; each XCD takes a contiguous
  // run of every round of tiles, odd rounds backwards.
  const int nx = gridDim.x >= 8 ? 8 : 1, per = gridDim.x / nx;
  if ((int)blockIdx.x >= per * nx) return;
  const int slot = (int)(blockIdx.x % nx) * per + (int)(blockIdx.x / nx), stride = per * nx;
  auto tile_at = [&](int round) -> int { return round * stride + ((round & 1) ? stride - 1 - slot : slot); };
  if (tile_at(0) >= total) return;       // a later round holds a tile for this workgroup only if the first was full

  // The load cursor: round and steps left of its tile, operands from its step
  // on, and how much of them may be read: K rows (operands with K outside) and
  // bytes (the others).
  int lround = 0, lk = 0, kleft = 0;
  const uint8_t *pa = nullptr, *pb = nullptr;
  int la = 0, lb = 0;
  uint32_t ca = 0, cb = 0;
  const uint32_t pitch_a = (uint32_t)(AT ? p.rows : p.k) * 2, pitch_b = (uint32_t)(BT ? p.n : p.k) * 2;

  // Tiles are numbered in blocks of 8 m-tiles x all n-tiles, n-major inside a
  // block, so that neighbours share operand rows; groups of the K form outermost.
  // Every wave writes the same ring entry and reads its own.
  auto plan = [&](int round) {
    int id = tile_at(round);
    Tile t{0, 0x7FFFFFFF, 0, 0, 0};
    la = lb = 0;
    kleft = 0;
    pa = pb = reinterpret_cast<const uint8_t*>(p.a);
    if (id < total) {
      const int plane = mt_total * nt, outer = AT ? id / plane : 0;
      id -= outer * plane;
      const int blk = id / (8 * nt), rem = id - blk * 8 * nt;
      const int rest = mt_total - blk * 8, mb = rest < 8 ? rest : 8;
      const int ni = rem / mb, mt = blk * 8 + (rem - ni * mb);
      t.n0 = (int64_t)ni * C::BN;
      const int64_t nn = p.n - t.n0 < C::BN ? p.n - t.n0 : C::BN;
      if constexpr (AT) {
        t.g = (int)ufirst((uint32_t)table.tiles[outer]);
        t.row0 = (int64_t)mt * C::BM;
        t.row_end = p.rows;
        const int64_t k0 = (int)ufirst((uint32_t)(t.g > 0 ? table.end[t.g - 1] : 0));
        const int64_t len = (int)ufirst((uint32_t)table.end[t.g]) - k0;
        t.nk = (int)((len + 63) / 64);
        pa = reinterpret_cast<const uint8_t*>(p.a + k0 * p.rows + t.row0);
        pb = reinterpret_cast<const uint8_t*>(p.b + k0 * p.n + t.n0);
        kleft = (int)len;
        ca = (uint32_t)t.row0 * 2;
        cb = (uint32_t)t.n0 * 2;
        if (len == 0) t.nk = 1;         // one step of zeros
      } else {
        // the group: how many tile counts are <= mt, in two reads of all lanes
        const int G = p.groups;
        int i0 = lane * 16 + 15;
        const int c1 = __popcll(__ballot(table.tiles[i0 < G ? i0 : G - 1] <= mt)) * 16;
        i0 = c1 + (lane & 15);
        const int c2 = __popcll(__ballot(lane < 16 && table.tiles[i0 < G ? i0 : G - 1] <= mt));
        t.g = (int)ufirst((uint32_t)(c1 + c2));
        const int before = t.g > 0 ? table.tiles[t.g - 1] : 0;
        const int64_t s = p.form == kMasked ? t.g * p.slot_rows : (int64_t)(t.g > 0 ? table.end[t.g - 1] : 0);
        t.row0 = ufirst64(s + (int64_t)(mt - before) * C::BM);
        t.row_end = (int)ufirst((uint32_t)table.end[t.g]);
        t.nk = (int)((p.k + 63) / 64);
        const int64_t mm = t.row_end - t.row0 < C::BM ? t.row_end - t.row0 : C::BM;
        pa = reinterpret_cast<const uint8_t*>(p.a + t.row0 * p.k);
        la = (int)ufirst((uint32_t)(mm * p.k * 2));
        pb = reinterpret_cast<const uint8_t*>(p.b + t.g * p.n * p.k + t.n0 * (BT ? 1 : p.k));
        lb = (int)ufirst((uint32_t)(nn * p.k * 2));
        kleft = (int)p.k;
        cb = (uint32_t)t.n0 * 2;
      }
    }
    lk = t.nk;
    if (lane == 0) ring[round % kRing] = t;
  };
  plan(0);

  // ---------------------------------------------------------------- loads
  const uint32_t lds0 = ufirst((uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)smem);
  uint32_t va[AL], vb[BL];
#pragma unroll
  for (int i = 0; i < AL; ++i) va[i] = load_offset<AT, C::BM>(i * C::WAVES + w, lane, pitch_a);
#pragma unroll
  for (int i = 0; i < BL; ++i) vb[i] = load_offset<BT, C::BN>(i * C::WAVES + w, lane, pitch_b);
  // row operands: the first K value of the lane's chunk (the swizzle does not
  // depend on i); bit 31 of an offset drops a chunk that lies past K
  const int chunk = ((lane & 7) ^ swz_row(w * 8 + (lane >> 3))) * 8;
  auto past_k = [&]() -> uint32_t { return AT || chunk < kleft ? 0u : 0x80000000u; };
  constexpr int kOps = AL + BL;
  // bytes of a step that may be read, from its first one
  auto limit = [&](bool t, int bytes, uint32_t pitch, uint32_t c) -> uint32_t {
    if (!t) return (uint32_t)bytes;
    return kleft <= 0 ? 0u : (uint32_t)(kleft < 64 ? kleft : 64) * pitch - c;
  };
  auto source_a = [&]() { return rsrc(pa, limit(AT, la, pitch_a, ca)); };
  auto source_b = [&]() { return rsrc(pb, limit(BT, lb, pitch_b, cb)); };
  // load l of an operand's step into the stage at stage_at
  auto load_a = [&](int l, const __amdgpu_buffer_rsrc_t& r, uint32_t stage_at, uint32_t past) {
    dma16(r, AT ? va[l] : va[l] | past, 0, stage_at + (uint32_t)(l * C::WAVES + w) * 1024);
  };
  auto load_b = [&](int l, const __amdgpu_buffer_rsrc_t& r, uint32_t stage_at, uint32_t past) {
    dma16(r, BT ? vb[l] : vb[l] | past, 0, stage_at + C::BM * 128 + (uint32_t)(l * C::WAVES + w) * 1024);
  };
  auto advance = [&]() {
    if (--lk == 0) {
      plan(++lround);
    } else {
      pa += AT ? (int64_t)pitch_a * 64 : 128;
      pb += BT ? (int64_t)pitch_b * 64 : 128;
      la = la - 128 > 0 ? la - 128 : 0;           // signed: a scalar maximum
      lb = lb - 128 > 0 ? lb - 128 : 0;
      kleft -= 64;
    }
  };
  for (int s = 0; s < ST; ++s) {
    const __amdgpu_buffer_rsrc_t rb0 = source_b(), ra0 = source_a();
    const uint32_t past = past_k();
#pragma unroll
    for (int l = 0; l < BL; ++l) load_b(l, rb0, lds0 + (uint32_t)s * C::STAGE, past);
#pragma unroll
    for (int l = 0; l < AL; ++l) load_a(l, ra0, lds0 + (uint32_t)s * C::STAGE, past);
    advance();
  }

  // ---------------------------------------------------------------- compute
  Frags<AT, C::BM, FI> fa;
  Frags<BT, C::BN, FJ> fb;
  fa.init(lane, wm * C::WTM);
  fb.init(lane, wn * C::WTN);
  v4f acc[FI][FJ];
  v4i ra[2][FI], rb[2][FJ];
  uint32_t stage = lds0;                 // of the current step
  auto fence = [&]() { __builtin_amdgcn_sched_barrier(0); };
  auto next_stage = [&]() { return stage + C::STAGE == lds0 + ST * C::STAGE ? lds0 : stage + C::STAGE; };
  // read number r of half ks of a step (B's, then A's), after read_from
  auto read_from = [&](int ks, uint32_t at) {
    fb.stage(at + C::BM * 128, ks);
    fa.stage(at, ks);
  };
  auto read1 = [&](int r, int ks) {
    if (r < FJ) rb[ks][r] = fb.read(r, ks);
    else ra[ks][r - FJ] = fa.read(r - FJ, ks);
  };
  constexpr int R = FI + FJ, G = FI * FJ;
  // A step's halves.  The products of half ks, with the reads of the next half
  // (of the stage at `at`) among them.  In the first half all of B has been read
  // when its fragments for the second are in registers: a barrier then frees its
  // part of the stage, and the loads of the step ST later go there; the second half
  // starts with the barrier that frees A's part, and has A's loads.  So the
  // loads are spread over the step, as the address unit needs them: bunched in
  // its second half they held the matrix instructions up.
  constexpr int kFreeB = G / 4;
  auto half = [&](auto ksc, uint32_t at, uint32_t freed) {
    constexpr int ks = decltype(ksc)::value;
    read_from(ks ^ 1, at);
    const uint32_t past = past_k();
    const __amdgpu_buffer_rsrc_t src = ks == 0 ? source_b() : source_a();
    each<G>([&](auto gc) {
      constexpr int g = decltype(gc)::value, i = g / FJ, j = g % FJ;
      if constexpr (ks == 0 && g == kFreeB) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        bar();
      }
      mfma<F16, C::BIG>(acc[i][j], rb[ks][j], ra[ks][i]);
      if constexpr (ks == 0) {
        each<FJ>([&](auto r) { if constexpr (r.value * kFreeB / 2 / FJ == g) read1(r.value, 1); });
        each<FI>([&](auto r) { if constexpr (kFreeB + r.value * (G / 2) / FI == g) read1(FJ + r.value, 1); });
        each<BL>([&](auto l) { if constexpr (kFreeB + l.value * (G - kFreeB) / BL == g) load_b(l.value, src, freed, past); });
      } else {
        each<R>([&](auto r) { if constexpr (r.value * (G / 2) / R == g) read1(r.value, 0); });
        each<AL>([&](auto l) { if constexpr (l.value * G / AL == g) load_a(l.value, src, freed, past); });
      }
      fence();
    });
  };

  // Wait states between matrix instructions and vector instructions that write
  // or read their sums: 19 cover the longest need of a 16 x 16 x 32 product.
  auto keep = [](v4f& v) {
    if constexpr (C::BIG) asm volatile("" : "+a"(v));
    else asm volatile("" : "+v"(v));
  };
  auto keep_all = [&]() {
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
      for (int j = 0; j < FJ; ++j) keep(acc[i][j]);
  };
  auto settle = [&]() {
    keep_all();
    fence();
    asm volatile("s_nop 15\n\ts_nop 2" ::: "memory");
    fence();
    keep_all();
  };

  wait_vm<(ST - 1) * kOps>();
  bar();
  read_from(0, stage);
#pragma unroll
  for (int r = 0; r < R; ++r) read1(r, 0);

  // the fewest stores of a tile, on top of the loads that may be under way
  constexpr int kStores = FI * 16 * C::WTN * 2 / 1024, kMost = (ST - 2) * kOps + BL + kStores;
  constexpr int kStoreWait = kMost < 63 ? kMost : 63;
  bool stored = false;
  for (int round = 0; tile_at(round) < total; ++round) {
    Tile t;
    {
      const Tile& v = ring[round % kRing];
      t.g = (int)ufirst((uint32_t)v.g);
      t.nk = (int)ufirst((uint32_t)v.nk);
      t.row0 = ufirst64(v.row0);
      t.row_end = ufirst64(v.row_end);
      t.n0 = ufirst64(v.n0);
    }
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
      for (int j = 0; j < FJ; ++j) acc[i][j] = v4f{};
    settle();
    for (int k = 0; k < t.nk; ++k) {
      half(std::integral_constant<int, 0>(), stage, stage);
      // this wave has read its stage, and the next step's has landed
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      // after a tile's stores, these may be under way too
      if (stored) wait_vm<kStoreWait>();
      else wait_vm<(ST - 2) * kOps + BL>();
      stored = false;
      bar();
      const uint32_t freed = stage;
      stage = next_stage();
      half(std::integral_constant<int, 1>(), stage, freed);
      advance();
    }
    settle();

    // ------------------------------------------------------------ epilogue
    // Through the wave's share of LDS, 16 rows at a time, so that stores write
    // whole lines: lane (x, q) holds columns 16 j + 4 q .. + 3 of row x.
    const int x = lane & 15, q = lane >> 4;
    uint8_t* mine = smem + ST * C::STAGE + w * C::ESHARE;
    const int64_t orow = AT ? (int64_t)t.g * p.rows : 0;
    // Stores past the tile's rows or the output's columns are dropped by the
    // buffer's end, not branched around: their number is known to the next wait.
    const uint32_t es = p.out_kind >= kOutF32 ? 4 : 2, opitch = (uint32_t)p.n * es;
    const int64_t rows = t.row_end - t.row0 < C::BM ? t.row_end - t.row0 : C::BM;
    const uint8_t* o0 = uniform(static_cast<const uint8_t*>(p.out) + ((orow + t.row0) * p.n + t.n0) * es);
    const __amdgpu_buffer_rsrc_t dst = rsrc(o0, ufirst((uint32_t)(rows * opitch - t.n0 * es)));
    auto store = [&](auto esc, auto addc, auto ntc) {
      constexpr int ES = decltype(esc)::value;
      constexpr int COLS = C::EROW / ES, PARTS = C::WTN / COLS, FP = FJ / PARTS;      // columns and fragments at a time
      constexpr int CH = C::EROW / 16, RPI = 64 / CH;                             // rows a store instruction
      const int lrow = lane / CH, ch = lane % CH;
#pragma unroll
      for (int i = 0; i < FI; ++i) {
#pragma unroll
        for (int part = 0; part < PARTS; ++part) {
#pragma unroll
          for (int j = 0; j < FP; ++j) {
            keep(acc[i][part * FP + j]);       // not read before its turn: there are no registers for all of them
            const v4f v = acc[i][part * FP + j];
            uint8_t* d = mine + x * C::ESTRIDE + (16 * j + 4 * q) * ES;
            if constexpr (ES == 2) *reinterpret_cast<uint2*>(d) = make_uint2(pack_half2<F16>(v[0], v[1]), pack_half2<F16>(v[2], v[3]));
            else *reinterpret_cast<v4f*>(d) = v;
          }
          fence();
          const int n = wn * C::WTN + part * COLS + ch * (16 / ES);
          const uint32_t off = (uint32_t)(wm * C::WTM + 16 * i + lrow) * opitch + (uint32_t)n * ES | (t.n0 + n < p.n ? 0u : 0x80000000u);
#pragma unroll
          for (int r = 0; r < 16 / RPI; ++r) {
            v4f v = *reinterpret_cast<const v4f*>(mine + (r * RPI + lrow) * C::ESTRIDE + ch * 16);
            const uint32_t at = off + (uint32_t)(r * RPI) * opitch;
            typedef unsigned int v4u __attribute__((ext_vector_type(4)));
            if constexpr (decltype(addc)::value)
              v += __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(dst, (int)at, 0, 0));
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, v), dst, (int)at, 0, decltype(ntc)::value ? 2 : 0);
          }
          fence();
        }
      }
    };
    constexpr std::true_type yes;
    constexpr std::false_type no;
    stored = true;
    if (p.out_kind == kOutF32Add) {
      // a group without rows adds nothing: its result is not even read (another stream may be adding to it)
      if (AT && ufirst((uint32_t)table.end[t.g]) == ufirst((uint32_t)(t.g > 0 ? table.end[t.g - 1] : 0))) stored = false;
      else store(std::integral_constant<int, 4>(), yes, no);
    }
    else if (p.out_kind == kOutF32 && p.stream) store(std::integral_constant<int, 4>(), no, yes);
    else if (p.out_kind == kOutF32) store(std::integral_constant<int, 4>(), no, no);
    else if (p.stream) store(std::integral_constant<int, 2>(), no, yes);
    else store(std::integral_constant<int, 2>(), no, no);
  }
  wait_vm<0>();       // no load may land in LDS after the workgroup has ended
}

}  // namespace half
}  // namespace hq
