// Low-rank adapters: v = x A[g]^T by place (shrink), out = base + scale[g] v
// B[g]^T by token (expand), and the gradients: u = dy B[g] (shrink), dx = base +
// scale[g] u A[g] (expand), dA = scale u^T x and dB = scale dy^T v (outer).
//
// Bound by bytes (large batches: x, base and out once each) and by latency (few
// tokens: chains of launches and dependent loads), never by products.  4096 tokens,
// 5120 -> 17408, 8 adapters of rank 64: 100 us, 3.5 TB/s (shrink 17, its slices' sum 5,
// expand 77); 64 tokens of 32 adapters of rank 16: 14.3 us (shrink 4.7, expand 9); 1
// token, 5120 -> 5120: 10.2 us in one launch.  Gradients of 16384 tokens, 4096 ->
// 4096, 8 adapters of rank 16: 171 us (shrink 36, outer 67, expand 65, sum 7).
#include <atomic>
#include <type_traits>

#include "group_tiles.hpp"
#include "half_internal.hpp"
#include "half_math.hpp"
#include "tile_util.hpp"

namespace hq {
namespace {

extern __shared__ __attribute__((aligned(16))) uint8_t smem[];

__device__ __forceinline__ int64_t token_at(const LoraPlan& pl, int place) {
  const int64_t t = pl.row_pair != nullptr ? pl.row_pair[place] : place;
  return t >= 0 && t < pl.m ? t : -1;
}
__device__ __forceinline__ v4i load8(const uint16_t* p) { return *reinterpret_cast<const v4i*>(p); }

// ------------------------------------------------------------------ shrink
constexpr int kShrinkWaves = 8;

// Few places an adapter: partial sums of a workgroup, 16 places x 16 RF ranks over
// one slice of K.  Its waves take blocks of 64 K values in turn, each lane loading
// its operands from memory (w [K, r]: through the wave's share of LDS, read
// transposed), and their sums meet in LDS in the order of the waves.
struct ShrinkArgs {
  LoraPlan pl;
  const uint16_t* z;       // [m, k]
  const uint16_t* w;       // [adapters, r, k]; WT: [adapters, k, r]
  float* out;              // [slices, max_rows, r]
  int k, r, slices;
};

template <bool F16, bool WT, int RF>
__global__ __launch_bounds__(kShrinkWaves * 64) void lora_shrink_few(ShrinkArgs p) {
  constexpr int W = kShrinkWaves, RN = 16 * RF, PITCH = RN * 2 + 16;
  constexpr int U = WT ? 1 : 2;                     // blocks in flight
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), x = lane & 15, q = lane >> 4;
  const int chunks = (p.r + RN - 1) / RN;
  int id = blockIdx.x;
  const int slice = id % p.slices;
  id /= p.slices;
  const int r0 = id % chunks * RN;
  const GroupTile t = group_tile(p.pl.group_end, p.pl.adapters, (int)p.pl.max_rows, 16, id / chunks);
  if (t.g < 0) return;
  const int place = t.row0 + x;
  const int64_t tok = place < t.row_end ? token_at(p.pl, place) : -1;
  const uint16_t* zp = p.z + (tok >= 0 ? tok : 0) * p.k + 8 * q;
  const uint16_t* wg = p.w + (int64_t)t.g * p.r * p.k;
  const uint16_t* wp[RF];
  if constexpr (!WT) {
#pragma unroll
    for (int j = 0; j < RF; ++j) {
      const int row = r0 + 16 * j + x;
      wp[j] = wg + (int64_t)(row < p.r ? row : p.r - 1) * p.k + 8 * q;
    }
  }
  uint8_t* mine = smem + w * 64 * PITCH;
  v4f acc[RF];
#pragma unroll
  for (int j = 0; j < RF; ++j) acc[j] = v4f{0, 0, 0, 0};
  const int blocks = (p.k + 63) / 64, last = blocks * (slice + 1) / p.slices;
  for (int b = blocks * slice / p.slices + w * U; b < last; b += W * U) {
    v4i zf[U][2], wf[U][2][RF];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k0 = (b + u) * 64;
      const bool on = b + u < last;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool in = on && k0 + 32 * h + 8 * q < p.k;
        zf[u][h] = v4i{0, 0, 0, 0};
        if (in && tok >= 0) zf[u][h] = load8(zp + k0 + 32 * h);
        if constexpr (!WT) {
#pragma unroll
          for (int j = 0; j < RF; ++j) {
            wf[u][h][j] = v4i{0, 0, 0, 0};
            if (in) wf[u][h][j] = load8(wp[j] + k0 + 32 * h);
          }
        }
      }
      if constexpr (WT) {
        // 64 rows of RN ranks: RN / 8 pieces of 16 bytes a lane
        v4i piece[2 * RF];
#pragma unroll
        for (int e = 0; e < 2 * RF; ++e) {
          const int c = lane + 64 * e, row = c / (2 * RF), col = c % (2 * RF) * 8;
          piece[e] = v4i{0, 0, 0, 0};
          if (k0 + row < p.k && r0 + col < p.r) piece[e] = load8(wg + (int64_t)(k0 + row) * p.r + r0 + col);
        }
#pragma unroll
        for (int e = 0; e < 2 * RF; ++e) {
          const int c = lane + 64 * e, row = c / (2 * RF), col = c % (2 * RF) * 8;
          *reinterpret_cast<v4i*>(mine + row * PITCH + col * 2) = piece[e];
        }
        asm volatile("" ::: "memory");
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < RF; ++j) {
            const uint8_t* at = mine + (32 * h + 8 * q + (x >> 2)) * PITCH + (16 * j + 4 * (x & 3)) * 2;
            wf[u][h][j] = join(read_transposed(at), read_transposed(at + 4 * PITCH));
          }
        asm volatile("" ::: "memory");
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < RF; ++j) acc[j] = product16<F16>(wf[u][h][j], zf[u][h], acc[j]);
  }
  v4f* part = reinterpret_cast<v4f*>(smem);         // [W][RF][64]
  __syncthreads();
#pragma unroll
  for (int j = 0; j < RF; ++j) part[(w * RF + j) * 64 + lane] = acc[j];
  __syncthreads();
  if (w >= RF) return;
  v4f s = part[w * 64 + lane];
#pragma unroll
  for (int e = 1; e < W; ++e) s += part[(e * RF + w) * 64 + lane];
  const int rank = r0 + 16 * w + 4 * q;
  if (tok >= 0 && rank < p.r) *reinterpret_cast<v4f*>(p.out + ((int64_t)slice * p.pl.max_rows + place) * p.r + rank) = s;
}

// Many: 64 places x 16 RF ranks over one slice of K.  Steps of 64 K values come
// straight into one of kManyStages LDS stages, three ahead of the products: a row's
// 128 bytes from its token's own address, chunks XOR-swizzled; w from a buffer
// that ends with it (ranks past r are not stored; values past K are zeros, and
// z's then any of the row's).  WT: w's rows are ranks of one K value, and its fragments
// are read transposed.  A wave has 16 places and all the ranks.
constexpr int kManyStages = 4;
template <int RF>
struct ShrinkStage {
  static constexpr int Z = 64 * 128, W = 16 * RF * 128, BYTES = Z + W;
  static constexpr int WL = RF < 2 ? 1 : RF / 2, OPS = 2 + WL;          // loads of w, and all, of a wave
};
template <bool F16, bool WT, int RF>
__global__ __launch_bounds__(256) void lora_shrink_many(ShrinkArgs p) {
  using namespace blk;
  using S = ShrinkStage<RF>;
  constexpr int RN = 16 * RF, ST = kManyStages;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), x = lane & 15, q = lane >> 4;
  const int chunks = (p.r + RN - 1) / RN;
  int id = blockIdx.x;
  const int slice = id % p.slices;
  id /= p.slices;
  const int r0 = id % chunks * RN;
  const GroupTile t = group_tile(p.pl.group_end, p.pl.adapters, (int)p.pl.max_rows, 64, id / chunks);
  if (t.g < 0) return;
  const int blocks = (p.k + 63) / 64, first = blocks * slice / p.slices, steps = blocks * (slice + 1) / p.slices - first;
  const uint32_t lds0 = ufirst((uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)smem);

  // z: load i fills rows (4 i + w) 8 .. + 7, lane j the chunk that belongs at slot j % 8 of row j / 8
  const int chunk = (lane & 7) ^ ((w * 8 + (lane >> 3)) >> 1 & 7);
  const uint16_t* zrow[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int place = t.row0 + (4 * i + w) * 8 + (lane >> 3);
    const int64_t tok = place < t.row_end ? token_at(p.pl, place) : -1;
    zrow[i] = p.z + (tok >= 0 ? tok : 0) * p.k;
  }
  // w: NT rows of 128 bytes, as z; WT 64 rows of RN ranks, 2 RF pieces each
  const uint8_t* wbase = reinterpret_cast<const uint8_t*>(p.w + (int64_t)t.g * p.r * p.k) + (WT ? r0 * 2 : (int64_t)r0 * p.k * 2);
  const uint32_t pitch = (uint32_t)(WT ? p.r : p.k) * 2;
  uint32_t woff[S::WL];
  int wld[S::WL];                        // the load's number
#pragma unroll
  for (int i = 0; i < S::WL; ++i) {
    wld[i] = RF == 1 ? w & 1 : 4 * i + w;
    if constexpr (WT) {
      const int piece = wld[i] * 64 + lane;
      woff[i] = (uint32_t)(piece / (2 * RF)) * pitch + (uint32_t)(piece % (2 * RF)) * 16;
    } else {
      const int row = wld[i] * 8 + (lane >> 3);
      woff[i] = (uint32_t)row * pitch + (uint32_t)(((lane & 7) ^ (row >> 1 & 7)) * 16);
    }
  }
  int wchunk[S::WL];
#pragma unroll
  for (int i = 0; i < S::WL; ++i) wchunk[i] = (lane & 7) ^ ((wld[i] * 8 + (lane >> 3)) >> 1 & 7);
  auto issue = [&](int step) {
    const int k0 = (first + step) * 64, kleft = step < steps ? p.k - k0 : 0;
    const uint32_t at = lds0 + (uint32_t)(step % ST) * S::BYTES;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      dma16_at(zrow[i] + (chunk * 8 < kleft ? k0 + chunk * 8 : 0), at + (uint32_t)(4 * i + w) * 1024);
    const uint8_t* b = wbase + (WT ? (int64_t)k0 * pitch : k0 * 2);
    // bytes to the end of w's adapter, of at most 64 rows (NT: RN)
    const int64_t rest = (WT ? (int64_t)(kleft < 64 ? kleft : 64) * pitch - r0 * 2
                             : (int64_t)(p.r - r0 < RN ? p.r - r0 : RN) * pitch - k0 * 2);
    const __amdgpu_buffer_rsrc_t src = rsrc(uniform(b), kleft > 0 ? ufirst((uint32_t)rest) : 0u);
#pragma unroll
    for (int i = 0; i < S::WL; ++i)
      dma16(src, WT || wchunk[i] * 8 < kleft ? woff[i] : 0x80000000u, 0, ufirst(at + S::Z + (uint32_t)wld[i] * 1024));
  };
#pragma unroll 1
  for (int s = 0; s < ST - 1; ++s) issue(s);

  v4f acc[RF];
#pragma unroll
  for (int j = 0; j < RF; ++j) acc[j] = v4f{0, 0, 0, 0};
  for (int s = 0; s < steps; ++s) {
    // this step has landed for every wave, and all have read the one before
    wait_vm<(ST - 2) * S::OPS>();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    bar();
    issue(s + ST - 1);
    const uint8_t* at = smem + (s % ST) * S::BYTES;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const v4i zf = *reinterpret_cast<const v4i*>(at + (16 * w + x) * 128 + (((4 * h + q) ^ (x >> 1 & 7)) << 4));
#pragma unroll
      for (int j = 0; j < RF; ++j) {
        v4i wf;
        if constexpr (WT) {
          const uint8_t* b = at + S::Z + (32 * h + 8 * q + (x >> 2)) * RN * 2 + (16 * j + 4 * (x & 3)) * 2;
          wf = join(read_transposed(b), read_transposed(b + 4 * RN * 2));
        } else {
          wf = *reinterpret_cast<const v4i*>(at + S::Z + (16 * j + x) * 128 + (((4 * h + q) ^ (x >> 1 & 7)) << 4));
        }
        acc[j] = product16<F16>(wf, zf, acc[j]);
      }
    }
    asm volatile("" ::: "memory");
  }
  wait_vm<0>();           // no load may land in LDS after the workgroup has ended
  const int place = t.row0 + 16 * w + x;
  if (place >= t.row_end || token_at(p.pl, place) < 0) return;
#pragma unroll
  for (int j = 0; j < RF; ++j) {
    const int rank = r0 + 16 * j + 4 * q;
    if (rank < p.r) *reinterpret_cast<v4f*>(p.out + ((int64_t)slice * p.pl.max_rows + place) * p.r + rank) = acc[j];
  }
}

// The sum of the slices' partial sums, in order, for every place with a token: those
// from the last end on have none, whatever token_at says (without a map it knows only
// m), and no partial sums.  The sums are read before the token and the ends have
// come (they lie in the workspace either way) and only the store waits for them.
__global__ __launch_bounds__(256) void lora_slices(LoraPlan pl, const float* part, int r, int slices, float* out) {
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, all = pl.max_rows * r;
  const int place = (int)(at / r);
  v4f v[16];
#pragma unroll
  for (int e = 0; e < 16; ++e)
    if (e < slices && at < all) v[e] = *reinterpret_cast<const v4f*>(part + e * all + at);
  const int last = last_end(pl.group_end, pl.adapters, (int)pl.max_rows);       // by whole waves
  if (at >= all || place >= last || token_at(pl, place) < 0) return;
  v4f s = v[0];
#pragma unroll
  for (int e = 1; e < 16; ++e)
    if (e < slices) s += v[e];
  *reinterpret_cast<v4f*>(out + at) = s;
}

// ------------------------------------------------------------------ expand
constexpr int kThreads = 256;

struct ExpandArgs {
  LoraPlan pl;
  const float* v;          // [slices, max_rows, r]
  const uint16_t* w;       // [adapters, n, r]; WT: [adapters, r, n]
  const uint16_t* base;
  uint16_t* out;           // [m, n]
  float* v_out;            // the slices' sums (nullptr: not kept)
  int n, r, slices;
  int chunk, chunks;       // columns of a workgroup, a multiple of 256
  unsigned tiles, rest;    // workgroups of places, of tokens without an adapter
  int rest_chunks;
};
constexpr int kRestRows = 64, kRestCols = 2048;

// Tokens without an adapter: base's row, or zeros.  A workgroup: 64 tokens, whose
// places its waves look up a lane each, and a share of the columns.
__device__ __forceinline__ void expand_rest(const ExpandArgs& p, int id) {
  const int c0 = id % p.rest_chunks * kRestCols;
  const int64_t t0 = (int64_t)(id / p.rest_chunks) * kRestRows;
  const int last = last_end(p.pl.group_end, p.pl.adapters, (int)p.pl.max_rows);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  bool none = false;
  if (t0 + lane < p.pl.m) {
    const int64_t place = p.pl.row_map != nullptr ? p.pl.row_map[t0 + lane] : t0 + lane;
    none = place < 0 || place >= last;
  }
  // every fourth of them is this wave's; four at a time, or the loads' latency of each adds up
  uint64_t all = __ballot(none), mine = 0;
  for (int i = 0; all != 0; ++i, all &= all - 1)
    if ((i & 3) == wave) mine |= all & -all;
  constexpr int ROWS = 4, PIECES = kRestCols / 512;
  while (mine != 0) {
    int64_t at[ROWS];                    // -1: no row
#pragma unroll
    for (int i = 0; i < ROWS; ++i, mine &= mine - 1) at[i] = mine != 0 ? (t0 + __builtin_ctzll(mine)) * p.n : -1;
    v4i v[ROWS][PIECES];
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
#pragma unroll
      for (int e = 0; e < PIECES; ++e) {
        const int col = c0 + lane * 8 + 512 * e;
        v[i][e] = v4i{0, 0, 0, 0};
        if (p.base != nullptr && at[i] >= 0 && col < p.n) v[i][e] = load8(p.base + at[i] + col);
      }
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
#pragma unroll
      for (int e = 0; e < PIECES; ++e) {
        const int col = c0 + lane * 8 + 512 * e;
        if (at[i] >= 0 && col < p.n) *reinterpret_cast<v4i*>(p.out + at[i] + col) = v[i][e];
      }
  }
}

// The values v scale of a wave's 16 places as fragments: each is kept as hi + lo, and
// 16 ranks' hi and 16 ranks' lo are the 32 K values of a matrix product with
// the ranks' weights twice (lanes q < 2: hi, the others: lo, of ranks 16 s + 8 (q % 2)
// .. + 7).  BF16: hi is the value cut to 8 bits, lo the rest rounded.  FP16: a
// place's values are first scaled by the power of two that takes its largest to
// [2^14, 2^15), undone in FP32 at the end, so that neither part leaves FP16's range.
// SL: slices read at once; HALVES: each half of the wave reads every other slice.
template <bool F16, int STEPS, int SL, bool HALVES = false>
struct Places {
  v4i part[STEPS];
  float factor, back;      // the place's power of two, and the one that undoes it
  int place;
  int64_t tok;             // -1: none

  __device__ __forceinline__ void find(const ExpandArgs& p, const GroupTile& t, int place0) {
    place = place0 + (threadIdx.x & 15);
    tok = place < t.row_end ? token_at(p.pl, place) : -1;
    factor = back = 1.0f;
  }
  // v of ranks 16 (s0 + s) + 8 (q % 2) .. + 7
  __device__ __forceinline__ void fetch(const ExpandArgs& p, int s0, v4f (&v)[STEPS][2]) const {
    const int h = (threadIdx.x >> 4) & 1;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) v[s][0] = v[s][1] = v4f{0, 0, 0, 0};
    const int each = HALVES ? 2 : 1;
    for (int e = HALVES ? (threadIdx.x >> 5) & 1 : 0; e < p.slices; e += SL * each) {
      v4f in[SL][STEPS][2];
#pragma unroll
      for (int i = 0; i < SL; ++i)
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
          in[i][s][0] = in[i][s][1] = v4f{0, 0, 0, 0};
          const int rank = 16 * (s0 + s) + 8 * h;
          if (tok >= 0 && rank < p.r && e + i * each < p.slices) {
            const v4f* src = reinterpret_cast<const v4f*>(p.v + ((int64_t)(e + i * each) * p.pl.max_rows + place) * p.r + rank);
            in[i][s][0] = src[0];
            in[i][s][1] = src[1];
          }
        }
#pragma unroll
      for (int i = 0; i < SL; ++i)
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
          v[s][0] += in[i][s][0];
          v[s][1] += in[i][s][1];
        }
    }
    if constexpr (HALVES) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[s][e >> 2][e & 3] += __shfl_xor(v[s][e >> 2][e & 3], 32, 64);
    }
  }
  // FP16: takes these ranks into the place's largest value
  __device__ __forceinline__ void largest(const v4f (&v)[STEPS][2], float scale, uint32_t& top) const {
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t a = __float_as_uint(v[s][e >> 2][e & 3] * scale) & 0x7fffffffu;
        top = a > top ? a : top;
      }
  }
  __device__ __forceinline__ void set_factor(uint32_t top) {
    const uint32_t o = (uint32_t)__shfl_xor((int)top, 16, 64);           // the other half of the ranks
    top = o > top ? o : top;
    int e = (int)(top >> 23);                                            // biased exponent
    e = e < 15 ? 15 : (e > 254 ? 141 : e);                               // Inf and NaN: unscaled
    factor = __uint_as_float((uint32_t)(127 + 141 - e) << 23);
    back = __uint_as_float((uint32_t)(127 - 141 + e) << 23);
  }
  __device__ __forceinline__ void split(const v4f (&v)[STEPS][2], float scale) {
    const bool low = (threadIdx.x & 32) != 0;
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float a = v[s][e >> 1][2 * (e & 1)] * scale, b = v[s][e >> 1][2 * (e & 1) + 1] * scale;
        uint32_t hi, lo;
        if constexpr (F16) {
          const float fa = a * factor, fb = b * factor;
          hi = pack_half2<true>(fa, fb);
          const float ha = f16_lo(hi), hb = f16_hi(hi);
          lo = pack_half2<true>(__builtin_fabsf(ha) == INFINITY ? 0.0f : fa - ha, __builtin_fabsf(hb) == INFINITY ? 0.0f : fb - hb);
        } else {
          hi = (__float_as_uint(a) >> 16) | (__float_as_uint(b) & 0xffff0000u);
          if (a != a) hi |= 0x7fc0u;                                     // a NaN whose top bits are an infinity's
          if (b != b) hi |= 0x7fc00000u;
          lo = pack_half2<false>(bf16_rest(a, bf16_cut(a)), bf16_rest(b, bf16_cut(b)));
        }
        part[s][e] = (int)(low ? lo : hi);
      }
  }
  // the fragments of the ranks from 16 s0 on
  __device__ __forceinline__ void load(const ExpandArgs& p, float scale, int s0) {
    v4f v[STEPS][2];
    fetch(p, s0, v);
    split(v, scale);
  }
  // FP16: the factor, and all fragments where the ranks are no more than STEPS hold
  __device__ __forceinline__ void start(const ExpandArgs& p, float scale, bool keep_v) {
    v4f v[STEPS][2];
    uint32_t top = 0;
    for (int s0 = 0; 16 * s0 < p.r; s0 += STEPS) {
      fetch(p, s0, v);
      if constexpr (F16) largest(v, scale, top);
      if (keep_v && tok >= 0 && (threadIdx.x & 32) == 0) {
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
          const int rank = 16 * (s0 + s) + 8 * ((threadIdx.x >> 4) & 1);
          if (rank < p.r) {
            v4f* d = reinterpret_cast<v4f*>(p.v_out + (int64_t)place * p.r + rank);
            d[0] = v[s][0];
            d[1] = v[s][1];
          }
        }
      }
    }
    if constexpr (F16) set_factor(top);
    if (p.r <= 16 * STEPS) split(v, scale);
  }
};

// Eight results of a lane.
template <bool F16>
__device__ __forceinline__ v4i expand_result(v4i base, v4f a, v4f b, float back) {
  const float f[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  v4i o;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t u = (uint32_t)base[e];
    o[e] = (int)pack_half2<F16>(__builtin_fmaf(f[2 * e], back, half_lo<F16>(u)),
                                __builtin_fmaf(f[2 * e + 1], back, half_hi<F16>(u)));
  }
  return o;
}

// Lanes of two neighbouring places trade a for b, so that what each had for 64
// neighbouring columns of its own row becomes 32 columns of the even place's row and
// 32 of the odd one's, and eight lanes a whole line of 128 bytes; and back again.
__device__ __forceinline__ void trade(bool odd, v4i& a, v4i& b) {
  const v4i mine = odd ? a : b;
  v4i other;
#pragma unroll
  for (int e = 0; e < 4; ++e) other[e] = __builtin_amdgcn_mov_dpp(mine[e], 0xB1, 0xf, 0xf, false);   // quad_perm:[1,0,3,2]
  if (odd) a = other;
  else b = other;
}

// The columns of fragment j of a lane's pairs: 32 (j / 2) + 8 (x / 4) + 4 (j % 2) + x %
// 4, so that a pair's sums are eight neighbouring columns 32 (j / 2) + 8 q .. + 7.
__device__ __forceinline__ int pair_column(int j, int x) { return 32 * (j >> 1) + 8 * (x >> 2) + 4 * (j & 1) + (x & 3); }

// Few places an adapter: a workgroup has 16 of them, each wave 64 of every 256
// columns, with the weights straight from memory (WT: through the wave's share of
// LDS, 64 ranks at a time, read transposed).
constexpr int kFewPitch = 144;
template <bool F16, bool WT, int STEPS>
__device__ __forceinline__ void expand_few(const ExpandArgs& p, int id) {
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), x = lane & 15, q = lane >> 4;
  const GroupTile t = group_tile(p.pl.group_end, p.pl.adapters, (int)p.pl.max_rows, 16, id / p.chunks);
  if (t.g < 0) return;
  const int c0 = id % p.chunks * p.chunk, c1 = c0 + p.chunk < p.n ? c0 + p.chunk : p.n;
  const float scale = p.pl.scale != nullptr ? p.pl.scale[t.g] : 1.0f;
  uint8_t* wt = smem + w * 16 * STEPS * kFewPitch;
  const uint16_t* wg = p.w + (int64_t)t.g * p.r * p.n;
  Places<F16, STEPS, STEPS == 4 ? 2 : 4, true> pl;
  pl.find(p, t, t.row0);
  v4i base[2], wf[STEPS][4];
  auto fetch = [&](int n0, int s0) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        wf[s][j] = v4i{0, 0, 0, 0};
        if constexpr (WT) {
          // 16 rows of 64 columns: 8 lanes a row, two loads; the others are not used
          const int row = 16 * (s0 + s) + (lane >> 3) + 8 * j, col = n0 + (lane & 7) * 8;
          if (j < 2 && row < p.r && col < c1) wf[s][j] = load8(wg + (int64_t)row * p.n + col);
        } else {
          const int col = n0 + pair_column(j, x), rank = 16 * (s0 + s) + 8 * (q & 1);
          if (rank < p.r) wf[s][j] = load8(wg + (int64_t)(col < c1 ? col : c1 - 1) * p.r + rank);
        }
      }
  };
  // base and results by whole lines, as expand_many has them
  const bool odd = x & 1;
  const int64_t other = __shfl_xor((long long)pl.tok, 1, 64);
  const int64_t tok[2] = {odd ? other : pl.tok, odd ? pl.tok : other};
  auto fetch_base = [&](int n0) {
    const int col = n0 + 32 * odd + 8 * q;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      base[h] = v4i{0, 0, 0, 0};
      if (p.base != nullptr && tok[h] >= 0 && col < c1) base[h] = load8(p.base + tok[h] * p.n + col);
    }
  };
  pl.start(p, scale, p.v_out != nullptr && c0 == 0 && w == 0);
  const int first = c0 + w * 64;
  if (first < c1) {
    fetch(first, 0);
    fetch_base(first);
  }
  for (int n0 = first; n0 < c1; n0 += 256) {
    v4f acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = v4f{0, 0, 0, 0};
    for (int s0 = 0; 16 * s0 < p.r; s0 += STEPS) {
      if (p.r > 16 * STEPS) pl.load(p, scale, s0);
      if constexpr (WT) {
        asm volatile("" ::: "memory");
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<v4i*>(wt + (16 * s + (lane >> 3) + 8 * e) * kFewPitch + (lane & 7) * 16) = wf[s][e];
        asm volatile("" ::: "memory");
      }
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v4i f = wf[s][j];
          if constexpr (WT) {
            const uint8_t* at = wt + (16 * s + 8 * (q & 1) + (x >> 2)) * kFewPitch + (32 * (j >> 1) + 8 * (x & 3) + 4 * (j & 1)) * 2;
            f = join(read_transposed(at), read_transposed(at + 4 * kFewPitch));
          }
          acc[j] = product16<F16>(f, pl.part[s], acc[j]);
        }
      if (16 * (s0 + STEPS) < p.r) fetch(n0, s0 + STEPS);
      else if (n0 + 256 < c1) fetch(n0 + 256, 0);
    }
    trade(odd, base[0], base[1]);
    v4i o[2] = {expand_result<F16>(base[0], acc[0], acc[1], pl.back), expand_result<F16>(base[1], acc[2], acc[3], pl.back)};
    trade(odd, o[0], o[1]);
    const int col = n0 + 32 * odd + 8 * q;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (tok[h] >= 0 && col < c1) *reinterpret_cast<v4i*>(p.out + tok[h] * p.n + col) = o[h];
    if (n0 + 256 < c1) fetch_base(n0 + 256);
  }
}

// Many places: a workgroup has 64 of them, 16 a wave, and goes through its columns
// 256 at a time, so that a row's loads and stores are 512 bytes.  The weights of a
// block of columns (and of 16 STEPS ranks) lie in one of two LDS buffers, which
// the waves fill together from registers that the next block's are loaded into
// meanwhile.
template <bool WT, int STEPS>
struct ManyCfg {
  static constexpr int SS = STEPS < 2 ? STEPS : 2;         // steps of a stage
  static constexpr int PITCH = WT ? 528 : SS * 32 + 16;
  static constexpr int BUF = WT ? 16 * SS * PITCH : 256 * PITCH;
};
template <bool F16, bool WT, int STEPS>
__device__ __forceinline__ void expand_many(const ExpandArgs& p, int id) {
  using M = ManyCfg<WT, STEPS>;
  constexpr int PITCH = M::PITCH, SS = M::SS, PCS = 2 * SS;         // PCS: 16-byte pieces of a thread
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), x = lane & 15, q = lane >> 4;
  const GroupTile t = group_tile(p.pl.group_end, p.pl.adapters, (int)p.pl.max_rows, 64, id / p.chunks);
  if (t.g < 0) return;
  const int c0 = id % p.chunks * p.chunk, c1 = c0 + p.chunk < p.n ? c0 + p.chunk : p.n;
  const float scale = p.pl.scale != nullptr ? p.pl.scale[t.g] : 1.0f;
  const uint16_t* wg = p.w + (int64_t)t.g * p.r * p.n;
  v4i piece[PCS];
  auto fetch = [&](int n0, int s0) {
#pragma unroll
    for (int e = 0; e < PCS; ++e) {
      const int c = tid + 256 * e;
      piece[e] = v4i{0, 0, 0, 0};
      if constexpr (WT) {
        const int row = 16 * s0 + (c >> 5), col = n0 + (c & 31) * 8;
        if (row < p.r && col < c1) piece[e] = load8(wg + (int64_t)row * p.n + col);
      } else {
        const int col = n0 + c / PCS, rank = 16 * s0 + c % PCS * 8;
        if (rank < p.r && col < c1) piece[e] = load8(wg + (int64_t)col * p.r + rank);
      }
    }
  };
  fetch(c0, 0);
  Places<F16, STEPS, STEPS == 4 ? 1 : 2> pl;
  pl.find(p, t, t.row0 + 16 * w);
  pl.start(p, scale, p.v_out != nullptr && c0 == 0);
  // the even and the odd place's tokens, and the lane's columns of both (jp even: one pair of 64)
  const bool odd = x & 1;
  const int64_t other = __shfl_xor((long long)pl.tok, 1, 64);
  const int64_t first = odd ? other : pl.tok, second = odd ? pl.tok : other;
  auto column = [&](int n0, int jp) { return n0 + 32 * ((jp & ~1) + odd) + 8 * q; };
  int buf = 0;
  for (int n0 = c0; n0 < c1; n0 += 256) {
    v4i base[8];                         // traded
#pragma unroll
    for (int jp = 0; jp < 8; ++jp) {
      const int64_t tok = jp & 1 ? second : first;
      base[jp] = v4i{0, 0, 0, 0};
      if (p.base != nullptr && tok >= 0 && column(n0, jp) < c1) base[jp] = load8(p.base + tok * p.n + column(n0, jp));
    }
    v4f acc[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[j] = v4f{0, 0, 0, 0};
    for (int s0 = 0; 16 * s0 < p.r; s0 += STEPS) {
      if (p.r > 16 * STEPS) pl.load(p, scale, s0);
#pragma unroll
      for (int s1 = 0; s1 < STEPS; s1 += SS) {
        if (16 * (s0 + s1) >= p.r) break;
        uint8_t* b = smem + buf * M::BUF;
        buf ^= 1;
#pragma unroll
        for (int e = 0; e < PCS; ++e) {
          const int c = tid + 256 * e;
          *reinterpret_cast<v4i*>(b + (WT ? (c >> 5) * PITCH + (c & 31) * 16 : c / PCS * PITCH + c % PCS * 16)) = piece[e];
        }
        if (16 * (s0 + s1 + SS) < p.r) fetch(n0, s0 + s1 + SS);
        else if (n0 + 256 < c1) fetch(n0 + 256, 0);
        // the buffer is written; its readers of two stages ago are past the barrier in between
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
#pragma unroll
        for (int s = 0; s < SS; ++s)
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            v4i wf;
            if constexpr (WT) {
              const uint8_t* at = b + (16 * s + 8 * (q & 1) + (x >> 2)) * PITCH + (32 * (j >> 1) + 8 * (x & 3) + 4 * (j & 1)) * 2;
              wf = join(read_transposed(at), read_transposed(at + 4 * PITCH));
            } else {
              wf = *reinterpret_cast<const v4i*>(b + pair_column(j, x) * PITCH + s * 32 + (q & 1) * 16);
            }
            acc[j] = product16<F16>(wf, pl.part[s1 + s], acc[j]);
            if (j % 8 == 7) __builtin_amdgcn_sched_barrier(0);       // no more fragments under way than registers hold
          }
      }
    }
#pragma unroll
    for (int jp = 0; jp < 8; jp += 2) {
      trade(odd, base[jp], base[jp + 1]);
      v4i a = expand_result<F16>(base[jp], acc[2 * jp], acc[2 * jp + 1], pl.back);
      v4i b = expand_result<F16>(base[jp + 1], acc[2 * jp + 2], acc[2 * jp + 3], pl.back);
      trade(odd, a, b);
      const int col = column(n0, jp);
      if (first >= 0 && col < c1) *reinterpret_cast<v4i*>(p.out + first * p.n + col) = a;
      if (second >= 0 && col < c1) *reinterpret_cast<v4i*>(p.out + second * p.n + col) = b;
    }
  }
}

template <bool F16, bool WT, int STEPS, bool MANY>
__global__ __launch_bounds__(kThreads, 2) void lora_expand(ExpandArgs p) {
  if (blockIdx.x >= p.tiles) expand_rest(p, (int)(blockIdx.x - p.tiles));
  else if constexpr (MANY) expand_many<F16, WT, STEPS>(p, (int)blockIdx.x);
  else expand_few<F16, WT, STEPS>(p, (int)blockIdx.x);
}

// ------------------------------------------------------------------ both at once
// A few places and little to read: one launch.  Every workgroup has 16 places
// and 1024 columns, 64 a wave; its 16 waves sum x A^T over all of K first, as
// lora_shrink_few does it, and each takes the sums from LDS as its places' values.
constexpr int kOneWaves = 16;
template <bool F16, int STEPS>
__global__ __launch_bounds__(kOneWaves * 64) void lora_one(ShrinkArgs a, ExpandArgs p) {
  constexpr int W = kOneWaves, RF = STEPS, U = STEPS == 1 ? 5 : 2, VP = 16 * RF + 4;
  if (blockIdx.x >= p.tiles) {
    if (threadIdx.x < 256) expand_rest(p, (int)(blockIdx.x - p.tiles));
    return;
  }
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), x = lane & 15, q = lane >> 4;
  const int id = (int)blockIdx.x;
  const GroupTile t = group_tile(p.pl.group_end, p.pl.adapters, (int)p.pl.max_rows, 16, id / p.chunks);
  if (t.g < 0) return;
  const float scale = p.pl.scale != nullptr ? p.pl.scale[t.g] : 1.0f;
  Places<F16, STEPS, 1> pl;
  pl.find(p, t, t.row0);
  const uint16_t* zp = a.z + (pl.tok >= 0 ? pl.tok : 0) * a.k + 8 * q;
  const uint16_t* wp[RF];
#pragma unroll
  for (int j = 0; j < RF; ++j) {
    const int row = 16 * j + x;
    wp[j] = a.w + ((int64_t)t.g * a.r + (row < a.r ? row : a.r - 1)) * a.k + 8 * q;
  }
  v4f sum[RF];
#pragma unroll
  for (int j = 0; j < RF; ++j) sum[j] = v4f{0, 0, 0, 0};
  for (int k0 = w * U * 64; k0 < a.k; k0 += W * U * 64) {
    v4i zf[U][2], wf[U][2][RF];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = k0 + u * 64 + h * 32;
#pragma unroll
        for (int j = 0; j < RF; ++j) {
          wf[u][h][j] = v4i{0, 0, 0, 0};
          if (at + 8 * q < a.k) wf[u][h][j] = load8(wp[j] + at);
        }
      }
    // after A's, which do not wait for the tokens to be looked up
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = k0 + u * 64 + h * 32;
        zf[u][h] = v4i{0, 0, 0, 0};
        if (at + 8 * q < a.k && pl.tok >= 0) zf[u][h] = load8(zp + at);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < RF; ++j) sum[j] = product16<F16>(wf[u][h][j], zf[u][h], sum[j]);
  }
  // the weights and the base of the wave's columns are on their way while the sums meet
  const int c0 = id % p.chunks * (W * 64), n0 = c0 + w * 64;
  const uint16_t* wg = p.w + (int64_t)t.g * p.r * p.n;
  v4i base[2], wf[STEPS][4];
#pragma unroll
  for (int jp = 0; jp < 2; ++jp) {
    const int col = n0 + 32 * jp + 8 * q;
    base[jp] = v4i{0, 0, 0, 0};
    if (p.base != nullptr && pl.tok >= 0 && col < p.n) base[jp] = load8(p.base + pl.tok * p.n + col);
  }
#pragma unroll
  for (int s = 0; s < STEPS; ++s)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = n0 + pair_column(j, x), rank = 16 * s + 8 * (q & 1);
      wf[s][j] = v4i{0, 0, 0, 0};
      if (rank < p.r && col < p.n) wf[s][j] = load8(wg + (int64_t)col * p.r + rank);
    }
  v4f* part = reinterpret_cast<v4f*>(smem);         // [W][RF][64]
  float* vs = reinterpret_cast<float*>(smem + W * RF * 1024);      // [16][VP]
#pragma unroll
  for (int j = 0; j < RF; ++j) part[(w * RF + j) * 64 + lane] = sum[j];
  __syncthreads();
  if (w < RF) {
    v4f s = part[w * 64 + lane];
#pragma unroll
    for (int e = 1; e < W; ++e) s += part[(e * RF + w) * 64 + lane];
    *reinterpret_cast<v4f*>(vs + x * VP + 16 * w + 4 * q) = s;
  }
  __syncthreads();
  v4f v[STEPS][2];
  uint32_t top = 0;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int rank = 16 * s + 8 * (q & 1);
    const bool on = pl.tok >= 0 && rank < p.r;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      v[s][e] = on ? *reinterpret_cast<const v4f*>(vs + x * VP + rank + 4 * e) : v4f{0, 0, 0, 0};
      if (p.v_out != nullptr && on && c0 == 0 && w == 0 && q < 2)
        *reinterpret_cast<v4f*>(p.v_out + (int64_t)pl.place * p.r + rank + 4 * e) = v[s][e];
    }
  }
  if constexpr (F16) {
    pl.largest(v, scale, top);
    pl.set_factor(top);
  }
  pl.split(v, scale);
  v4f acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    acc[j] = v4f{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < STEPS; ++s) acc[j] = product16<F16>(wf[s][j], pl.part[s], acc[j]);
  }
#pragma unroll
  for (int jp = 0; jp < 2; ++jp) {
    const int col = n0 + 32 * jp + 8 * q;
    if (pl.tok >= 0 && col < p.n)
      *reinterpret_cast<v4i*>(p.out + pl.tok * p.n + col) =
          expand_result<F16>(base[jp], acc[2 * jp], acc[2 * jp + 1], pl.back);
  }
}

// ------------------------------------------------------------------ outer
// One chunk of an adapter's places: part[chunk] = sum over them of u[place, i]
// z[token, j], 16 RF ranks i and 256 columns j a workgroup, a wave 64 columns.  32
// places at a time: z's rows and u, cut into three BF16 parts that hold all its
// 24 bits, lie in LDS and are read transposed; FP16's z is cut into two BF16
// parts when it is read, and the products of the least parts (2^-24 of the
// value) left out.
struct OuterArgs {
  LoraPlan pl;
  const float* u;          // [slices, max_rows, r]
  const uint16_t* z;       // [m, k]
  float* part;             // [chunks, r, k]; UT: [chunks, k, r]
  float* out;              // [adapters, r, k]; UT: [adapters, k, r]
  int k, r, slices;
  int places;              // of a chunk
  unsigned tiles;          // workgroups
  bool accumulate;
};
constexpr int kOuterCols = 256, kOuterRows = 32;

// The scale of adapter g's sums.  One that is not finite counts only where one of its
// places holds a token: the gradients of an adapter without tokens are zeros, and 0
// times an infinity or NaN is not.  Uniform arguments, all lanes of the wave.
__device__ __forceinline__ float sum_scale(const LoraPlan& pl, int g, int row0, int row_end) {
  const float f = pl.scale != nullptr ? pl.scale[g] : 1.0f;
  if (__builtin_fabsf(f) < INFINITY) return f;
  bool any = false;
  for (int place = row0 + (int)(threadIdx.x & 63); place < row_end && !any; place += 64) any = token_at(pl, place) >= 0;
  return __ballot(any) != 0 ? f : 0.0f;
}

template <int RF>
constexpr int outer_smem() { return kOuterRows * (kOuterCols * 2 + 16) + 3 * kOuterRows * (RF * 32 + 16); }

template <bool F16, bool UT, int RF>
__device__ __forceinline__ void outer_tile(const OuterArgs& p, int id) {
  constexpr int ZP = kOuterCols * 2 + 16, UP = RF * 32 + 16;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), x = lane & 15, q = lane >> 4;
  const int kt = (p.k + kOuterCols - 1) / kOuterCols, rt = (p.r + 16 * RF - 1) / (16 * RF);
  const int j0 = id % kt * kOuterCols;
  id /= kt;
  const int i0 = id % rt * 16 * RF;
  const GroupTile t = group_tile(p.pl.group_end, p.pl.adapters, (int)p.pl.max_rows, p.places, id / rt);
  if (t.g < 0) return;
  const int end = t.row0 + p.places < t.row_end ? t.row0 + p.places : t.row_end;
  uint8_t* zt = smem;
  uint8_t* ut = smem + kOuterRows * ZP;
  v4f acc[RF][4];
#pragma unroll
  for (int i = 0; i < RF; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0, 0, 0, 0};
  // a thread's pieces: 32 lanes a row of z (4 pieces), 4 RF lanes a row of u (four values each)
  constexpr int UE = (RF + 1) / 2;
  v4i zr[4];
  v4f ur[UE];
  // their places' tokens are looked up a step before
  int64_t tz[4], tu[UE];
  auto look = [&](int place0) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int place = place0 + (tid >> 5) + 8 * e;
      tz[e] = place < end ? token_at(p.pl, place) : -1;
    }
#pragma unroll
    for (int e = 0; e < UE; ++e) {
      const int c = tid + 256 * e, place = place0 + c / (4 * RF);
      tu[e] = c < 128 * RF && place < end ? token_at(p.pl, place) : -1;
    }
  };
  auto fetch = [&](int place0) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int col = j0 + (tid & 31) * 8;
      zr[e] = v4i{0, 0, 0, 0};
      if (tz[e] >= 0 && col < p.k) zr[e] = load8(p.z + tz[e] * p.k + col);
    }
#pragma unroll
    for (int e = 0; e < UE; ++e) {
      const int c = tid + 256 * e, place = place0 + c / (4 * RF), rank = i0 + c % (4 * RF) * 4;
      const float* src = p.u + (int64_t)place * p.r + rank;
      ur[e] = v4f{0, 0, 0, 0};
      for (int s = 0; s < p.slices; s += 4) {
        v4f in[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          in[i] = v4f{0, 0, 0, 0};
          if (tu[e] >= 0 && rank < p.r && s + i < p.slices)
            in[i] = *reinterpret_cast<const v4f*>(src + (int64_t)(s + i) * p.pl.max_rows * p.r);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) ur[e] += in[i];
      }
    }
  };
  look(t.row0);
  fetch(t.row0);
  look(t.row0 + kOuterRows);
  for (int place0 = t.row0; place0 < end; place0 += kOuterRows) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) *reinterpret_cast<v4i*>(zt + ((tid >> 5) + 8 * e) * ZP + (tid & 31) * 16) = zr[e];
#pragma unroll
    for (int e = 0; e < UE; ++e) {
      const int c = tid + 256 * e;
      if (c >= 128 * RF) break;
      uint8_t* d = ut + c / (4 * RF) * UP + c % (4 * RF) * 8;
      float v[4] = {ur[e][0], ur[e][1], ur[e][2], ur[e][3]};
#pragma unroll
      for (int part = 0; part < 3; ++part) {
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h[i] = __float_as_uint(v[i]) >> 16;
          if (v[i] != v[i]) h[i] |= 0x7fc0u;
          v[i] = bf16_rest(v[i], bf16_cut(v[i]));
        }
        *reinterpret_cast<uint2*>(d + part * kOuterRows * UP) = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
      }
    }
    __syncthreads();
    if (place0 + kOuterRows < end) {
      fetch(place0 + kOuterRows);
      look(place0 + 2 * kOuterRows);
    }
    const int row = 8 * q + (x >> 2);
    v4i uf[RF][3];
#pragma unroll
    for (int i = 0; i < RF; ++i)
#pragma unroll
      for (int part = 0; part < 3; ++part) {
        const uint8_t* at = ut + (part * kOuterRows + row) * UP + (16 * i + 4 * (x & 3)) * 2;
        uf[i][part] = join(read_transposed(at), read_transposed(at + 4 * UP));
      }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint8_t* at = zt + row * ZP + (64 * w + 16 * j + 4 * (x & 3)) * 2;
      v4i zf = join(read_transposed(at), read_transposed(at + 4 * ZP)), zl = v4i{0, 0, 0, 0};
      if constexpr (F16) {
        const v8h v = __builtin_bit_cast(v8h, zf);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = (float)v[2 * e], b = (float)v[2 * e + 1], ca = bf16_cut(a), cb = bf16_cut(b);
          uint32_t hi = (__float_as_uint(a) >> 16) | (__float_as_uint(b) & 0xffff0000u);
          if (a != a) hi |= 0x7fc0u;
          if (b != b) hi |= 0x7fc00000u;
          zf[e] = (int)hi;
          zl[e] = (int)pack_half2<false>(bf16_rest(a, ca), bf16_rest(b, cb));
        }
      }
#pragma unroll
      for (int i = 0; i < RF; ++i) {
        auto mul = [&](v4i u, v4i z) {
          acc[i][j] = UT ? product16<false>(u, z, acc[i][j]) : product16<false>(z, u, acc[i][j]);
        };
        if constexpr (F16) {
          mul(uf[i][1], zl);
          mul(uf[i][0], zl);
        }
        mul(uf[i][2], zf);
        mul(uf[i][1], zf);
        mul(uf[i][0], zf);
      }
    }
  }
  // an adapter's only chunk is its result; else lora_sum joins them
  const bool whole = t.index == t.first && t.row_end - t.row0 <= p.places, add = whole && p.accumulate;
  const float f = whole ? sum_scale(p.pl, t.g, t.row0, t.row_end) : 1.0f;
  float* out = (whole ? p.out + (int64_t)t.g * p.r * p.k : p.part + (int64_t)t.index * p.r * p.k);
  // four neighbours of a lane: columns (rank x) or, UT, ranks (column x)
#pragma unroll
  for (int i = 0; i < RF; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int rank = i0 + 16 * i + (UT ? 4 * q : x), col = j0 + 64 * w + 16 * j + (UT ? x : 4 * q);
      if (rank >= p.r || col >= p.k) continue;
      v4f* d = reinterpret_cast<v4f*>(out + (UT ? (int64_t)col * p.r + rank : (int64_t)rank * p.k + col));
      v4f v = acc[i][j];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= f;
      if (add) v += *d;
      *d = v;
    }
}

// dA's and dB's chunks in one launch; where they are few, dx's tiles too (its
// registers would keep the chunks from filling the chip; three workgroups a compute
// unit where 16 ranks allow it: 2918 tokens, 1568 + 1344 wide, 33.0 -> 28.6 us, while
// dx alone is better off with two, 4096 places of 17408 columns 76 us against 81; the
// bound costs lora_back<., 1, true> four to six spilled registers, inside that gain).
struct BackArgs {
  OuterArgs da, db;
  ExpandArgs dx;
};
template <bool F16, int RF>
__global__ __launch_bounds__(kThreads) void lora_outer(BackArgs p) {
  if (blockIdx.x < p.da.tiles) outer_tile<F16, false, RF>(p.da, (int)blockIdx.x);
  else outer_tile<F16, true, RF>(p.db, (int)(blockIdx.x - p.da.tiles));
}
template <bool F16, int RF, bool MANY>
__global__ __launch_bounds__(kThreads, RF == 1 ? 3 : 2) void lora_back(BackArgs p) {
  unsigned id = blockIdx.x;
  if (id < p.da.tiles) return outer_tile<F16, false, RF>(p.da, (int)id);
  id -= p.da.tiles;
  if (id < p.db.tiles) return outer_tile<F16, true, RF>(p.db, (int)id);
  id -= p.db.tiles;
  if (id >= p.dx.tiles) return expand_rest(p.dx, (int)(id - p.dx.tiles));
  if constexpr (MANY) expand_many<F16, true, RF>(p.dx, (int)id);
  else expand_few<F16, true, RF>(p.dx, (int)id);
}

// da, db: scale times the sum of an adapter's chunks, in order, where it has several;
// zeros where it has none.
struct SumArgs {
  LoraPlan pl;
  const float *pa, *pb;
  float *da, *db;
  int64_t na, nb;          // values of an adapter
  int places;
  unsigned blocks;         // of an adapter
  bool accumulate;
};
__global__ __launch_bounds__(kThreads) void lora_sum(SumArgs p) {
  const int g = (int)(blockIdx.x / p.blocks);
  const int64_t at = ((int64_t)(blockIdx.x % p.blocks) * kThreads + threadIdx.x) * 4;
  const GroupTile t = group_tile<true>(p.pl.group_end, p.pl.adapters, (int)p.pl.max_rows, p.places, g);
  const int chunks = (t.row_end - t.row0 + p.places - 1) / p.places;
  if (chunks == 1 || (p.accumulate && chunks == 0)) return;
  const float f = chunks > 0 ? sum_scale(p.pl, g, t.row0, t.row_end) : 0.0f;      // by whole waves
  if (at >= p.na + p.nb) return;
  const bool b = at >= p.na;
  const int64_t n = b ? p.nb : p.na, i = b ? at - p.na : at;
  v4f* out = reinterpret_cast<v4f*>((b ? p.db : p.da) + g * n + i);
  const float* src = (b ? p.pb : p.pa) + t.first * n + i;
  v4f s = {0, 0, 0, 0};
  for (int c = 0; c < chunks; ++c) s += *reinterpret_cast<const v4f*>(src + c * n);
#pragma unroll
  for (int e = 0; e < 4; ++e) s[e] *= f;
  if (p.accumulate) s += *out;
  *out = s;
}

// ------------------------------------------------------------------ plans
int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }
// At most this many tiles of bm places.
int64_t tile_bound(int64_t max_rows, int64_t adapters, int64_t bm) {
  return max_rows / bm + (max_rows < adapters ? max_rows : adapters);
}
constexpr int64_t kFill = 512;           // workgroups that fill the chip

// Few places an adapter on average: tiles of 16, more of 64.  The average is over all
// adapters, since only the device knows which of them have tokens: 1000 tokens of two
// adapters, 4096 x 4096, take 25.4 us with 64 adapters of rank 64 loaded and 19.4 with two
// (5120 x 5120, rank 16: 14.3 and 15.8).
struct ShrinkPlan {
  bool many;
  int rf, slices;
  int64_t tiles;                         // of places
  bool summed() const { return many && slices > 1 && (slices > 4 || rf == 4); }      // by lora_slices; else by the readers
};
ShrinkPlan shrink_plan(int64_t max_rows, int64_t adapters, int64_t k, int64_t r) {
  ShrinkPlan p{max_rows > 16 * adapters, r <= 16 ? 1 : r <= 32 ? 2 : 4, 1, 0};
  p.tiles = tile_bound(max_rows, adapters, p.many ? 64 : 16);
  const int64_t wgs = p.tiles * up(r, 16 * p.rf), most = up(k, p.many ? 512 : 64 * kShrinkWaves);
  int64_t s = wgs > 0 ? (p.many && p.rf < 4 ? 2 * kFill : kFill) / wgs : 1;
  s = s < most ? s : most;
  p.slices = (int)(s < 1 ? 1 : s > 16 ? 16 : s);
  return p;
}
// Places of a workgroup: 16 where an adapter has few on average, else 64.
int expand_places(int64_t max_rows, int64_t adapters) { return max_rows <= 16 * adapters ? 16 : 64; }
// Steps of 16 ranks whose fragments a wave keeps.
int expand_steps(int64_t r) { return r <= 16 ? 1 : r <= 32 ? 2 : 4; }
// Columns of a workgroup: what makes about 2 kFill workgroups, whole 256s.
int expand_chunk(int64_t tiles, int64_t n) {
  const int64_t across = tiles > 0 ? up(2 * kFill, tiles) : 1;
  return (int)(up(up(n, across), 256) * 256);
}
int outer_rf(int64_t r) { return r <= 16 ? 1 : r <= 32 ? 2 : 4; }
// Places of a chunk of dA and dB: about 2 kFill workgroups.
int outer_places(int64_t max_rows, int64_t n, int64_t k, int64_t r) {
  const int64_t across = (up(n, kOuterCols) + up(k, kOuterCols)) * up(r, 16 * outer_rf(r));
  int64_t p = up(up(max_rows * across, 2 * kFill), 64) * 64;
  return (int)(p < 128 ? 128 : p > 8192 ? 8192 : p);
}

// More than 64 KB of dynamic LDS, allowed once per device (twice is harmless).
template <class K>
hipError_t allow_smem(K kernel, int bytes, std::atomic<bool> (&set)[64]) {
  if (bytes <= 65536) return hipSuccess;
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const bool cached = dev >= 0 && dev < 64;
  if (cached && set[dev].load(std::memory_order_acquire)) return hipSuccess;
  e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess && cached) set[dev].store(true, std::memory_order_release);
  return e;
}

template <bool F16, bool WT, int RF>
hipError_t shrink_rf(hipStream_t s, const ShrinkArgs& p, const ShrinkPlan& plan) {
  const int64_t wgs = plan.tiles * up(p.r, 16 * RF) * p.slices;
  if (plan.many) {
    constexpr int bytes = kManyStages * ShrinkStage<RF>::BYTES;
    static std::atomic<bool> set[64];
    const hipError_t e = allow_smem(lora_shrink_many<F16, WT, RF>, bytes, set);
    if (e != hipSuccess || wgs == 0) return e;
    hipLaunchKernelGGL((lora_shrink_many<F16, WT, RF>), dim3((unsigned)wgs), dim3(256), bytes, s, p);
  } else {
    constexpr int kSum = kShrinkWaves * RF * 1024, kW = WT ? kShrinkWaves * 64 * (RF * 32 + 16) : 0;
    constexpr int bytes = kSum > kW ? kSum : kW;
    static std::atomic<bool> set[64];
    const hipError_t e = allow_smem(lora_shrink_few<F16, WT, RF>, bytes, set);
    if (e != hipSuccess || wgs == 0) return e;
    hipLaunchKernelGGL((lora_shrink_few<F16, WT, RF>), dim3((unsigned)wgs), dim3(kShrinkWaves * 64), bytes, s, p);
  }
  return hipGetLastError();
}
// z w^T into `out` [max_rows, r], or, where the plan leaves the slices to the
// readers, [slices, max_rows, r]; `parts` holds the slices where they are summed here.
template <bool F16, bool WT>
hipError_t shrink(hipStream_t s, const LoraPlan& pl, const uint16_t* z, const uint16_t* w, int64_t k, int64_t r,
                  const ShrinkPlan& plan, float* parts, float* out) {
  const ShrinkArgs p{pl, z, w, plan.summed() ? parts : out, (int)k, (int)r, plan.slices};
  const hipError_t e = plan.rf == 1   ? shrink_rf<F16, WT, 1>(s, p, plan)
                       : plan.rf == 2 ? shrink_rf<F16, WT, 2>(s, p, plan)
                                      : shrink_rf<F16, WT, 4>(s, p, plan);
  if (e != hipSuccess || !plan.summed()) return e;
  hipLaunchKernelGGL(lora_slices, dim3((unsigned)up(pl.max_rows * r, 1024)), dim3(256), 0, s, pl, parts, (int)r, plan.slices, out);
  return hipGetLastError();
}

ExpandArgs expand_args(const LoraPlan& pl, const float* v, const uint16_t* w, const uint16_t* base, uint16_t* out,
                       float* v_out, int64_t n, int64_t r, int slices) {
  ExpandArgs p{pl, v, w, base, out, v_out, (int)n, (int)r, slices, 0, 0, 0, 0, 0};
  const int64_t tiles = tile_bound(pl.max_rows, pl.adapters, expand_places(pl.max_rows, pl.adapters));
  p.chunk = expand_chunk(tiles, n);
  p.chunks = (int)up(n, p.chunk);
  p.tiles = (unsigned)(tiles * p.chunks);
  const int64_t rest = up(pl.m, kRestRows);
  p.rest_chunks = (int)up(n, kRestCols);
  p.rest = base != out ? (unsigned)(rest * p.rest_chunks) : 0;
  return p;
}

template <bool F16, bool WT, int STEPS, bool MANY>
hipError_t expand_one(hipStream_t s, const ExpandArgs& p) {
  constexpr int bytes = MANY ? 2 * ManyCfg<WT, STEPS>::BUF : WT ? 4 * 16 * STEPS * kFewPitch : 0;
  static std::atomic<bool> set[64];
  const hipError_t e = allow_smem(lora_expand<F16, WT, STEPS, MANY>, bytes, set);
  if (e != hipSuccess || p.tiles + p.rest == 0) return e;
  hipLaunchKernelGGL((lora_expand<F16, WT, STEPS, MANY>), dim3(p.tiles + p.rest), dim3(kThreads), bytes, s, p);
  return hipGetLastError();
}
template <bool F16, bool WT>
hipError_t expand(hipStream_t s, const ExpandArgs& p) {
  const bool many = expand_places(p.pl.max_rows, p.pl.adapters) == 64;
  switch (expand_steps(p.r)) {
    case 1: return many ? expand_one<F16, WT, 1, true>(s, p) : expand_one<F16, WT, 1, false>(s, p);
    case 2: return many ? expand_one<F16, WT, 2, true>(s, p) : expand_one<F16, WT, 2, false>(s, p);
    default: return many ? expand_one<F16, WT, 4, true>(s, p) : expand_one<F16, WT, 4, false>(s, p);
  }
}
// One launch does it: few places an adapter, ranks that a wave's registers hold (of
// 64 one launch takes 14.1 us where two take 12.7, of 32 10.4 and 13.2), no more
// workgroups than the chip takes at once, and an A that one compute unit reads in about
// a launch's time (every workgroup reads all of its adapter's; 16 ranks of 6000
// values 12.5 us, 13.3).
bool one_launch(const LoraPlan& pl, int64_t n, int64_t k, int64_t r) {
  return pl.max_rows <= 16 * pl.adapters && r <= 32 && r * k <= 3 << 15 &&
         tile_bound(pl.max_rows, pl.adapters, 16) * up(n, kOneWaves * 64) <= kFill / 2;
}
template <bool F16, int STEPS>
hipError_t one(hipStream_t s, const ShrinkArgs& a, const ExpandArgs& p) {
  constexpr int bytes = kOneWaves * STEPS * 1024 + 16 * (16 * STEPS + 4) * 4;
  static std::atomic<bool> set[64];
  const hipError_t e = allow_smem(lora_one<F16, STEPS>, bytes, set);
  if (e != hipSuccess || p.tiles + p.rest == 0) return e;
  hipLaunchKernelGGL((lora_one<F16, STEPS>), dim3(p.tiles + p.rest), dim3(kOneWaves * 64), bytes, s, a, p);
  return hipGetLastError();
}

template <bool F16>
hipError_t forward(hipStream_t s, const LoraArgs& p) {
  const LoraPlan& pl = p.plan;
  if (one_launch(pl, p.n, p.k, p.r)) {
    const ShrinkArgs a{pl, p.x, p.a, nullptr, (int)p.k, (int)p.r, 1};
    ExpandArgs x = expand_args(pl, nullptr, p.b, p.base, p.out, p.v, p.n, p.r, 1);
    x.chunk = kOneWaves * 64;
    x.chunks = (int)up(p.n, x.chunk);
    x.tiles = (unsigned)(tile_bound(pl.max_rows, pl.adapters, 16) * x.chunks);
    return p.r <= 16 ? one<F16, 1>(s, a, x) : one<F16, 2>(s, a, x);
  }
  const ShrinkPlan plan = shrink_plan(pl.max_rows, pl.adapters, p.k, p.r);
  // the workspace: the slices (if any), then v where it is not kept
  float* parts = static_cast<float*>(p.workspace);
  const bool several = plan.slices > 1 && !plan.summed();
  float* v = several ? parts : p.v != nullptr ? p.v : parts + (plan.summed() ? plan.slices * pl.max_rows * p.r : 0);
  const hipError_t e = shrink<F16, false>(s, pl, p.x, p.a, p.k, p.r, plan, parts, v);
  if (e != hipSuccess) return e;
  const ExpandArgs x = expand_args(pl, v, p.b, p.base, p.out, several ? p.v : nullptr, p.n, p.r, several ? plan.slices : 1);
  return expand<F16, false>(s, x);
}

// Floats of slices and sums of a shrink in the workspace.
uint64_t shrink_space(const ShrinkPlan& p, int64_t max_rows, int64_t r) {
  return (uint64_t)(p.slices + (p.summed() ? 1 : 0)) * max_rows * r;
}
uint64_t chunk_count(int64_t max_rows, int64_t n, int64_t k, int64_t r, int64_t adapters) {
  return (uint64_t)tile_bound(max_rows, adapters, outer_places(max_rows, n, k, r));
}

template <bool F16, int RF>
hipError_t outer(hipStream_t s, const BackArgs& p) {
  const unsigned wgs = p.da.tiles + p.db.tiles;
  if (wgs == 0) return hipSuccess;
  hipLaunchKernelGGL((lora_outer<F16, RF>), dim3(wgs), dim3(kThreads), outer_smem<RF>(), s, p);
  return hipGetLastError();
}
template <bool F16, int RF, bool MANY>
hipError_t back_one(hipStream_t s, const BackArgs& p) {
  constexpr int a = MANY ? 2 * ManyCfg<true, RF>::BUF : 4 * 16 * RF * kFewPitch, b = outer_smem<RF>(), bytes = a > b ? a : b;
  static std::atomic<bool> set[64];
  const hipError_t e = allow_smem(lora_back<F16, RF, MANY>, bytes, set);
  const unsigned wgs = p.da.tiles + p.db.tiles + p.dx.tiles + p.dx.rest;
  if (e != hipSuccess || wgs == 0) return e;
  hipLaunchKernelGGL((lora_back<F16, RF, MANY>), dim3(wgs), dim3(kThreads), bytes, s, p);
  return hipGetLastError();
}
template <bool F16, int RF>
hipError_t back(hipStream_t s, const BackArgs& p, const LoraPlan& pl) {
  const bool many = expand_places(pl.max_rows, pl.adapters) == 64;
  if (p.dx.out != nullptr && (int64_t)p.da.tiles + p.db.tiles + p.dx.tiles <= 2 * kFill)
    return many ? back_one<F16, RF, true>(s, p) : back_one<F16, RF, false>(s, p);
  const hipError_t e = outer<F16, RF>(s, p);
  return e != hipSuccess || p.dx.out == nullptr ? e : expand<F16, true>(s, p.dx);
}

template <bool F16>
hipError_t backward(hipStream_t s, const LoraArgs& p) {
  const LoraPlan& pl = p.plan;
  const ShrinkPlan plan = shrink_plan(pl.max_rows, pl.adapters, p.n, p.r);
  // the workspace: slices, u, then the chunks of dA and of dB
  float* parts = static_cast<float*>(p.workspace);
  float* u = parts + (plan.summed() ? plan.slices * pl.max_rows * p.r : 0);
  float* pa = parts + shrink_space(plan, pl.max_rows, p.r);
  float* pb = pa + chunk_count(pl.max_rows, p.n, p.k, p.r, pl.adapters) * p.r * p.k;
  const int slices = plan.summed() ? 1 : plan.slices;
  hipError_t e = shrink<F16, true>(s, pl, p.dy, p.b, p.n, p.r, plan, parts, u);
  if (e != hipSuccess) return e;
  const int places = outer_places(pl.max_rows, p.n, p.k, p.r);
  const int64_t each = tile_bound(pl.max_rows, pl.adapters, places) * up(p.r, 16 * outer_rf(p.r));
  BackArgs x;
  x.da = OuterArgs{pl, u, p.x, pa, p.da, (int)p.k, (int)p.r, slices, places, (unsigned)(each * up(p.k, kOuterCols)),
                   p.accumulate};
  x.db = OuterArgs{pl, p.v, p.dy, pb, p.db, (int)p.n, (int)p.r, 1, places, (unsigned)(each * up(p.n, kOuterCols)),
                   p.accumulate};
  x.dx = expand_args(pl, u, p.a, p.base, p.out, nullptr, p.k, p.r, slices);
  const int rf = outer_rf(p.r);
  e = rf == 1 ? back<F16, 1>(s, x, pl) : rf == 2 ? back<F16, 2>(s, x, pl) : back<F16, 4>(s, x, pl);
  if (e != hipSuccess) return e;
  SumArgs m{pl, pa, pb, p.da, p.db, p.r * p.k, p.r * p.n, places, (unsigned)up(p.r * (p.k + p.n), 4 * kThreads), p.accumulate};
  hipLaunchKernelGGL(lora_sum, dim3(m.blocks * (unsigned)pl.adapters), dim3(kThreads), 0, s, m);
  return hipGetLastError();
}

}  // namespace

// The most work items of a launch that the call makes.
int64_t lora_work_items(const LoraArgs& p, bool backward) {
  const LoraPlan& pl = p.plan;
  int64_t most = 0;
  auto launch = [&](int64_t wgs, int64_t threads) {
    const int64_t v = wgs < ((int64_t)1 << 40) ? wgs * threads : (int64_t)1 << 50;
    most = v > most ? v : most;
  };
  const int64_t inner = backward ? p.n : p.k, across = backward ? p.k : p.n;
  const int64_t rest = p.base != p.out ? up(pl.m, kRestRows) * up(across, kRestCols) : 0;
  if (!backward && one_launch(pl, p.n, p.k, p.r)) {
    launch(tile_bound(pl.max_rows, pl.adapters, 16) * up(p.n, kOneWaves * 64) + rest, kOneWaves * 64);
    return most;
  }
  const ShrinkPlan plan = shrink_plan(pl.max_rows, pl.adapters, inner, p.r);
  launch(plan.tiles * up(p.r, 16 * plan.rf) * plan.slices, plan.many ? 256 : kShrinkWaves * 64);
  if (plan.summed()) launch(up(pl.max_rows * p.r, 1024), 256);
  const int64_t tiles = tile_bound(pl.max_rows, pl.adapters, expand_places(pl.max_rows, pl.adapters));
  const int64_t expand = tiles * up(across, expand_chunk(tiles, across)) + rest;
  if (!backward) {
    launch(expand, kThreads);
    return most;
  }
  const int64_t chunks = tile_bound(pl.max_rows, pl.adapters, outer_places(pl.max_rows, p.n, p.k, p.r));
  const int64_t sums = chunks * up(p.r, 16 * outer_rf(p.r)) * (up(p.n, kOuterCols) + up(p.k, kOuterCols));
  const bool dx = p.out != nullptr, joint = dx && sums + expand - rest <= 2 * kFill;
  launch(joint ? sums + expand : sums, kThreads);
  if (dx && !joint) launch(expand, kThreads);
  launch(up(p.r * (p.k + p.n), 4 * kThreads) * pl.adapters, kThreads);
  return most;
}

uint64_t lora_workspace_bytes(int64_t max_rows, int64_t, int64_t k, int64_t r, int32_t adapters) {
  return 4 * shrink_space(shrink_plan(max_rows, adapters, k, r), max_rows, r);
}
uint64_t lora_backward_workspace_bytes(int64_t max_rows, int64_t n, int64_t k, int64_t r, int32_t adapters) {
  return 4 * (shrink_space(shrink_plan(max_rows, adapters, n, r), max_rows, r) +
              chunk_count(max_rows, n, k, r, adapters) * (uint64_t)(r * (k + n)));
}

hipError_t launch_lora(hipStream_t s, const LoraArgs& p) { return p.f16 ? forward<true>(s, p) : forward<false>(s, p); }
hipError_t launch_lora_backward(hipStream_t s, const LoraArgs& p) {
  return p.f16 ? backward<true>(s, p) : backward<false>(s, p);
}

}  // namespace hq
