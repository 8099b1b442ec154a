// The tiled 16-bit GEMM kernel (half_gemm.hip picks the shape, half_tiled_*.hip
// instantiate it).
#pragma once

#include "block_gemm.hpp"
#include "half_internal.hpp"
#include "tile_util.hpp"

namespace hq {
namespace half {

using namespace blk;

typedef short v4s __attribute__((ext_vector_type(4)));

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

template <int BM_, int BN_, int WM_, int WN_, int ST_>
struct Cfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, ST = ST_;
  static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int WTM = BM / WM, WTN = BN / WN, FI = WTM / 16, FJ = WTN / 16;
  static constexpr int AL = BM / 8 / WAVES, BL = BN / 8 / WAVES;   // loads a wave, per step
  static constexpr int STAGE = (BM + BN) * 128;
  static constexpr bool AGPR = FI * FJ >= 64;        // sums that take half of the register file
  // the epilogue's share of a wave: 16 rows of at most 256 bytes, padded
  static constexpr int EROW = WTN * 2 < 256 ? WTN * 2 : 256, ESTRIDE = EROW + 16, ESHARE = 16 * ESTRIDE;
  static constexpr int SMEM = ST * STAGE + WAVES * ESHARE;
  static_assert(BM / 8 % WAVES == 0 && BN / 8 % WAVES == 0 && AL >= 1 && BL >= 1, "whole loads");
  static_assert(WAVES % 2 == 0, "the row swizzle's period");
};

struct Table {
  int end[kMaxGroups];     // rows where group g ends
  int tiles[kMaxGroups];   // inclusive count of m-tiles (row forms)
};

// Where a tile sits (uniform).
struct Tile {
  int g, nk;
  int64_t row0, row_end, n0;
};
constexpr int kRing = 16;

// LDS layouts of an operand's 64 K values.  ROW: 128-byte rows, 16-byte chunks
// XOR-swizzled.  COL (T): 64 rows of W columns, 32-byte pieces XOR-swizzled.
__device__ __forceinline__ int swz_row(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int swz_col(int krow) { return (krow & 3) | ((krow >> 3) & 1) << 2; }

// Source offset (bytes) of lane `lane` of the wave-load number `ld`.
template <bool T, int W>
__device__ __forceinline__ uint32_t load_offset(int ld, int lane, uint32_t pitch) {
  if constexpr (!T) {
    const int row = ld * 8 + (lane >> 3);
    return (uint32_t)row * pitch + (uint32_t)(((lane & 7) ^ swz_row(row)) << 4);
  } else {
    constexpr int CH = W / 8;                       // 16-byte chunks of a K row
    const int krow = ld * (64 / CH) + lane / CH, c = lane % CH;
    constexpr int MASK = W / 16 < 8 ? W / 16 - 1 : 7;
    return (uint32_t)krow * pitch + (uint32_t)(((((c >> 1) ^ (swz_col(krow) & MASK)) << 1 | (c & 1)) << 4));
  }
}

// Reads of the fragments (16 rows or columns x 32 K values) of a wave: lane (x, q)
// holds K values 8 q .. + 7 of row or column x.
template <bool T, int W, int F>
struct Frags {
  static constexpr int N = T ? F : 2;
  uint32_t off[N];       // ROW: by K half; COL: by fragment
  uint32_t at[N];        // the same in the stage that is read
  __device__ __forceinline__ void init(int lane, int wave_base) {
    const int x = lane & 15, q = lane >> 4;
    if constexpr (!T) {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) off[ks] = (uint32_t)((wave_base + x) * 128 + (((4 * ks + q) ^ swz_row(x)) << 4));
    } else {
      constexpr int MASK = W / 16 < 8 ? W / 16 - 1 : 7;
      const int krow = 8 * q + (x >> 2);
#pragma unroll
      for (int i = 0; i < F; ++i)
        off[i] = (uint32_t)(krow * 2 * W + (((wave_base / 16 + i) ^ (swz_col(krow) & MASK)) << 5) + 8 * (x & 3));
    }
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
__global__ __launch_bounds__(C::THREADS, C::WAVES / 4) void half_gemm_tiled(HalfGemmArgs p) {
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
  uint32_t la = 0, lb = 0, ca = 0, cb = 0, live = 0;
  const uint32_t pitch_a = (uint32_t)(AT ? p.rows : p.k) * 2, pitch_b = (uint32_t)(BT ? p.n : p.k) * 2;

  // Tiles are numbered in blocks of 8 m-tiles x all n-tiles, n-major inside a
  // block, so that neighbours share operand rows; groups of the K form outermost.
  // Every wave writes the same ring entry and reads its own.
  auto plan = [&](int round) {
    int id = tile_at(round);
    Tile t{0, 0x7FFFFFFF, 0, 0, 0};
    la = lb = live = 0;
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
        t.g = outer;
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
        la = ufirst((uint32_t)(mm * p.k * 2));
        pb = reinterpret_cast<const uint8_t*>(p.b + t.g * p.n * p.k + t.n0 * (BT ? 1 : p.k));
        lb = ufirst((uint32_t)(nn * p.k * 2));
        kleft = (int)p.k;
        cb = (uint32_t)t.n0 * 2;
        live = 128;
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
  // row operands: bit 31 drops the chunks past K of its last step (the swizzle does not depend on i)
  const uint32_t krem = (uint32_t)p.k & 63;
  const uint32_t drop = !AT && krem != 0 && (uint32_t)(((lane & 7) ^ swz_row(w * 8 + (lane >> 3))) * 8) >= krem ? 0x80000000u : 0u;
  constexpr int kOps = AL + BL;
  // bytes of a step that may be read, from its first one
  auto limit = [&](bool t, uint32_t bytes, uint32_t pitch, uint32_t c) -> uint32_t {
    if (!t) return bytes;
    return kleft <= 0 ? 0u : (uint32_t)(kleft < 64 ? kleft : 64) * pitch - c;
  };
  // load l (B's, then A's) of the cursor's step into the stage at stage_at
  auto issue1 = [&](int l, uint32_t stage_at) {
    const uint32_t mask = !AT && lk == 1 ? drop : 0u;
    if (l < BL) {
      const uint32_t v = BT ? vb[l] : vb[l] | mask;
      dma16(rsrc(pb, limit(BT, lb, pitch_b, cb)), v, 0, stage_at + C::BM * 128 + (uint32_t)(l * C::WAVES + w) * 1024);
    } else {
      const uint32_t v = AT ? va[l - BL] : va[l - BL] | mask;
      dma16(rsrc(pa, limit(AT, la, pitch_a, ca)), v, 0, stage_at + (uint32_t)((l - BL) * C::WAVES + w) * 1024);
    }
  };
  auto advance = [&]() {
    if (--lk == 0) {
      plan(++lround);
    } else {
      pa += AT ? (int64_t)pitch_a * 64 : 128;
      pb += BT ? (int64_t)pitch_b * 64 : 128;
      la -= live;
      lb -= live;
      kleft -= 64;
    }
  };
  for (int s = 0; s < ST; ++s) {
#pragma unroll
    for (int l = 0; l < kOps; ++l) issue1(l, lds0 + (uint32_t)s * C::STAGE);
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
  // read number r of the set `set` (B's, then A's), after read_from
  auto read_from = [&](int set, uint32_t at) {
    fb.stage(at + C::BM * 128, set);
    fa.stage(at, set);
  };
  auto read1 = [&](int r, int set) {
    if (r < FJ) rb[set][r] = fb.read(r, set);
    else ra[set][r - FJ] = fa.read(r - FJ, set);
  };
  constexpr int R = FI + FJ, G = FI * FJ;
  // the products of one set, with the reads of the other set (from `at`) and, for
  // set 1, the loads into the freed stage spread over them
  auto sub = [&](auto setc, uint32_t at, uint32_t freed) {
    constexpr int set = decltype(setc)::value;
    read_from(set ^ 1, at);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int i = g / FJ, j = g % FJ;
      mfma<F16, C::AGPR>(acc[i][j], rb[set][j], ra[set][i]);
#pragma unroll
      for (int r = g * R / G; r < (g + 1) * R / G; ++r) read1(r, set ^ 1);
      if constexpr (set == 1) {
#pragma unroll
        for (int l = g * kOps / G; l < (g + 1) * kOps / G; ++l) issue1(l, freed);
      }
      fence();
    }
  };

  // Wait states between matrix instructions and vector instructions that write
  // or read their sums: 19 cover the longest need of a 16 x 16 x 32 product.
  auto keep = [](v4f& v) {
    if constexpr (C::AGPR) asm volatile("" : "+a"(v));
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
      sub(std::integral_constant<int, 0>(), stage, 0);
      // the stage has been read by this wave; the next step's has landed
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      wait_vm<(ST - 2) * kOps>();
      bar();
      const uint32_t freed = stage;
      stage = next_stage();
      sub(std::integral_constant<int, 1>(), stage, freed);
      advance();
    }
    settle();

    // ------------------------------------------------------------ epilogue
    // Through the wave's share of LDS, 16 rows at a time, so that stores write
    // whole lines: lane (x, q) holds columns 16 j + 4 q .. + 3 of row x.
    const int x = lane & 15, q = lane >> 4;
    uint8_t* mine = smem + ST * C::STAGE + w * C::ESHARE;
    const int64_t wrow0 = t.row0 + wm * C::WTM, wn0 = t.n0 + wn * C::WTN;
    const int64_t orow = AT ? (int64_t)t.g * p.rows : 0;
    auto store = [&](auto esc, auto addc) {
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
          const int64_t n = wn0 + part * COLS + ch * (16 / ES);
#pragma unroll
          for (int r = 0; r < 16 / RPI; ++r) {
            v4f v = *reinterpret_cast<const v4f*>(mine + (r * RPI + lrow) * C::ESTRIDE + ch * 16);
            const int64_t row = wrow0 + 16 * i + r * RPI + lrow;
            if (row < t.row_end && n < p.n) {
              v4f* d = reinterpret_cast<v4f*>(static_cast<uint8_t*>(p.out) + ((orow + row) * p.n + n) * ES);
              if constexpr (decltype(addc)::value) v = *d + v;
              *d = v;
            }
          }
          fence();
        }
      }
    };
    if (p.out_kind == kOutF32) store(std::integral_constant<int, 4>(), std::false_type());
    else if (p.out_kind == kOutF32Add) store(std::integral_constant<int, 4>(), std::true_type());
    else store(std::integral_constant<int, 2>(), std::false_type());
  }
  wait_vm<0>();       // no load may land in LDS after the workgroup has ended
}

}  // namespace half
}  // namespace hq
